"""ctypes binding of libpaged_gqa.so (see ``include/paged_gqa.h`` and
``include/paged_gqa_serving.h``).

Argument marshalling only: every step of the attention runs in the CUDA
library.  torch supplies device memory and the current stream.  There is no
fallback: if the library is missing or no GPU is present, calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import sys
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
# PA_GQA_LIB names another build of the library (e.g. the checked build)
LIB_PATH = os.environ.get("PA_GQA_LIB") or os.path.join(PKG, "libpaged_gqa.so")

PA_F32, PA_F16, PA_BF16 = 0, 1, 2
DTYPE_CODE = {"f32": PA_F32, "f16": PA_F16, "bf16": PA_BF16}
PA_DEV_BAD_PAGE, PA_DEV_BAD_LEN, PA_DEV_TIMEOUT, PA_DEV_OOB = 1, 2, 4, 8
PA_DEV_NO_PAGES, PA_DEV_BAD_INDEX = 16, 32
PA_FORM_AUTO, PA_FORM_PAIR, PA_FORM_COUNTED = 0, 1, 2
STATUS = {0: "PA_OK", 1: "PA_ERR_NULL", 2: "PA_ERR_SHAPE", 3: "PA_ERR_DTYPE",
          4: "PA_ERR_ALIGN", 5: "PA_ERR_WORKSPACE", 6: "PA_ERR_UNSUPPORTED", 7: "PA_ERR_CUDA"}

EXPORTS = ("pa_params_init", "pa_status_string", "pa_decode_plan", "pa_decode_workspace_size",
           "pa_decode", "pa_decode_partial", "pa_combine", "pa_prefill_workspace_size",
           "pa_prefill_chunk", "pa_version", "pa_decode_append", "pa_decode_noalloc",
           "pa_build_flags", "pa_decode_kernels", "pa_rows_init", "pa_prompt",
           "pa_tree_workspace_size", "pa_tree", "pa_store", "pa_pages_workspace_size",
           "pa_pages_resize", "pa_pages_fork", "pa_pages_compact", "pa_pages_copy")


class PaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


class Params(ctypes.Structure):
    """Mirror of ``pa_params``."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("max_context_len", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("q_dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("deterministic", ctypes.c_int32),
                ("num_splits", ctypes.c_int32), ("decode_phases", ctypes.c_int32),
                ("decode_q_rows", ctypes.c_int32), ("sliding_window", ctypes.c_int32),
                ("decode_form", ctypes.c_int32), ("debug_timeout", ctypes.c_int32)]


class Rows(ctypes.Structure):
    """Mirror of ``pa_rows``."""
    _fields_ = [("total_rows", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("source_rows", ctypes.c_int32), ("mask_words", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Loads the library (raises if it was not built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: run paged_kv_gqa_02_gb300.build.build()")
            L = ctypes.CDLL(path)
            P = ctypes.POINTER(Params)
            vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            L.pa_params_init.argtypes = [P]
            L.pa_params_init.restype = P
            L.pa_status_string.argtypes = [ctypes.c_int]
            L.pa_status_string.restype = ctypes.c_char_p
            L.pa_decode_plan.argtypes = [P, ctypes.POINTER(i32), ctypes.POINTER(i32)]
            L.pa_decode_workspace_size.argtypes = [P]
            L.pa_decode_workspace_size.restype = sz
            L.pa_decode.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
            L.pa_decode_partial.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp]
            L.pa_decode_append.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
            L.pa_combine.argtypes = [P, vp, vp, i32, vp, vp, vp]
            L.pa_prefill_workspace_size.argtypes = [P, i32, i32]
            L.pa_prefill_workspace_size.restype = sz
            L.pa_prefill_chunk.argtypes = [P, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp]
            L.pa_decode_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
            if hasattr(L, "pa_decode_kernels"):
                L.pa_decode_kernels.argtypes = [P, i32]
                L.pa_decode_kernels.restype = i32
            for name in ("pa_decode_plan", "pa_decode", "pa_decode_append", "pa_decode_partial",
                         "pa_combine", "pa_prefill_chunk", "pa_decode_noalloc"):
                getattr(L, name).restype = ctypes.c_int
            R = ctypes.POINTER(Rows)
            L.pa_rows_init.argtypes = [R]
            L.pa_rows_init.restype = R
            L.pa_prompt.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp]
            L.pa_tree_workspace_size.argtypes = [P, R]
            L.pa_tree.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
            L.pa_store.argtypes = [P, R, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            L.pa_pages_workspace_size.argtypes = [P]
            L.pa_pages_resize.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp, vp]
            L.pa_pages_fork.argtypes = [P, vp, vp, vp, vp, vp, i32, vp, vp]
            L.pa_pages_compact.argtypes = [P, vp, vp, vp, vp, i32, vp, vp, sz, vp, vp]
            L.pa_pages_copy.argtypes = [P, vp, vp, vp, i32, vp, vp]
            for name in ("pa_tree_workspace_size", "pa_pages_workspace_size"):
                getattr(L, name).restype = sz
            for name in ("pa_prompt", "pa_tree", "pa_store", "pa_pages_resize", "pa_pages_fork",
                         "pa_pages_compact", "pa_pages_copy"):
                getattr(L, name).restype = ctypes.c_int
            L.pa_version.restype = i32
            if hasattr(L, "pa_build_flags"):
                L.pa_build_flags.restype = i32
            _lib = L
    return _lib


def make_params(*, num_seqs, num_q_heads, num_kv_heads, head_dim, page_size, num_pages,
                max_blocks_per_seq, max_context_len, scale=None, dtype="bf16", kv_dtype=None,
                deterministic=1, num_splits=0, strides=(0, 0, 0), decode_phases=0,
                decode_q_rows=0, sliding_window=0, decode_form=0, debug_timeout=0,
                out_dtype="f32") -> Params:
    p = Params()
    load().pa_params_init(ctypes.byref(p))
    p.num_seqs, p.num_q_heads, p.num_kv_heads = num_seqs, num_q_heads, num_kv_heads
    p.head_dim, p.page_size, p.num_pages = head_dim, page_size, num_pages
    p.max_blocks_per_seq, p.max_context_len = max_blocks_per_seq, max_context_len
    p.page_stride, p.token_stride, p.head_stride = strides
    p.scale = (1.0 / math.sqrt(head_dim)) if scale is None else scale
    p.q_dtype = DTYPE_CODE[dtype]
    p.kv_dtype = DTYPE_CODE[kv_dtype or dtype]
    p.out_dtype = DTYPE_CODE[out_dtype]
    p.deterministic, p.num_splits = deterministic, num_splits
    p.decode_phases = decode_phases
    p.decode_q_rows = decode_q_rows
    p.sliding_window = sliding_window
    p.decode_form = decode_form
    p.debug_timeout = debug_timeout
    return p


def params_for(wl, num_pages=None, **kw) -> Params:
    """Params of a ``workloads.Workload``."""
    args = dict(num_seqs=wl.num_seqs, num_q_heads=wl.num_q_heads, num_kv_heads=wl.num_kv_heads,
                head_dim=wl.head_dim, page_size=wl.page_size,
                num_pages=num_pages or wl.num_pages, max_blocks_per_seq=wl.max_blocks_per_seq,
                max_context_len=wl.max_blocks_per_seq * wl.page_size, scale=wl.scale,
                dtype=wl.q_dtype, kv_dtype=wl.kv_dtype)
    args.update(kw)
    return make_params(**args)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(code, what):
    if code != 0:
        raise PaError(code, what)


def decode_plan(p: Params):
    S, tok = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load().pa_decode_plan(ctypes.byref(p), ctypes.byref(S), ctypes.byref(tok)),
           "pa_decode_plan")
    return S.value, tok.value


def decode_kernels(p: Params, with_append: bool = False) -> int:
    """Kernels one pa_decode (or pa_decode_append) call launches (-1: invalid)."""
    return int(load().pa_decode_kernels(ctypes.byref(p), int(with_append)))


def decode_workspace_size(p: Params) -> int:
    return int(load().pa_decode_workspace_size(ctypes.byref(p)))


def prefill_workspace_size(p: Params, total_q: int, max_q_len: int) -> int:
    return int(load().pa_prefill_workspace_size(ctypes.byref(p), total_q, max_q_len))


def _empty_out(q, p):
    import torch
    return torch.empty((q.shape[0], p.num_q_heads, p.head_dim), dtype=torch.float32,
                       device=q.device)


def decode(p: Params, q, k_cache, v_cache, block_tables, context_lens, out=None,
           workspace=None, dev_status=None, stream=None):
    """Decode attention; q [B][Hq][D] -> out [B][Hq][D] f32 (torch CUDA tensors)."""
    import torch
    if out is None:
        out = _empty_out(q, p)
    if workspace is None:
        n = decode_workspace_size(p)
        workspace = torch.zeros(max(n, 1), dtype=torch.uint8, device=q.device) if n else None
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pa_decode(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                            _ptr(block_tables), _ptr(context_lens), _ptr(out), _ptr(workspace),
                            nbytes, _ptr(dev_status), _stream(stream)), "pa_decode")
    return out


def decode_append(p: Params, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, out=None,
                  workspace=None, dev_status=None, stream=None):
    """Decode with the new token's K/V ([B][Hkv][D]) written to row L-1 of each
    sequence's last page first; k_cache / v_cache are updated in place."""
    import torch
    if out is None:
        out = _empty_out(q, p)
    if workspace is None:
        n = decode_workspace_size(p)
        workspace = torch.zeros(max(n, 1), dtype=torch.uint8, device=q.device) if n else None
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pa_decode_append(ctypes.byref(p), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                   _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), _ptr(out),
                                   _ptr(workspace), nbytes, _ptr(dev_status), _stream(stream)),
           "pa_decode_append")
    return out


def decode_partial(p: Params, q, k_cache, v_cache, block_tables, context_lens, partial_ml,
                   partial_acc, num_splits, dev_status=None, stream=None):
    _check(load().pa_decode_partial(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_tables), _ptr(context_lens), _ptr(partial_ml),
                                    _ptr(partial_acc), num_splits, _ptr(dev_status),
                                    _stream(stream)), "pa_decode_partial")


def combine(p: Params, partial_ml, partial_acc, num_splits, out, stream=None, splits_per_seq=None):
    """pa_combine: num_splits is the partials' split stride (max_splits);
    splits_per_seq (device int32 [B], optional) limits each sequence."""
    _check(load().pa_combine(ctypes.byref(p), _ptr(partial_ml), _ptr(partial_acc), num_splits,
                             _ptr(splits_per_seq), _ptr(out), _stream(stream)), "pa_combine")
    return out


def prefill_chunk(p: Params, q, cu_q_lens, total_q, max_q_len, k_cache, v_cache, block_tables,
                  context_lens, out=None, workspace=None, dev_status=None, stream=None):
    """Chunked causal prefill; q [total_q][Hq][D] -> out [total_q][Hq][D] f32."""
    import torch
    if out is None:
        out = _empty_out(q, p)
    if workspace is None:
        n = prefill_workspace_size(p, total_q, max_q_len)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pa_prefill_chunk(ctypes.byref(p), _ptr(q), _ptr(cu_q_lens), total_q, max_q_len,
                                   _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                   _ptr(context_lens), _ptr(out), _ptr(workspace), nbytes,
                                   _ptr(dev_status), _stream(stream)), "pa_prefill_chunk")
    return out


# ---- numpy inputs -> torch device tensors ----------------------------------

def to_device(arr, dtype: str | None = None, device="cuda"):
    """numpy array (bf16 given as uint16 bits when dtype == 'bf16') -> torch."""
    import numpy as np
    import torch
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(arr).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(arr))
    return t.to(device)


def device_inputs(inp, wl_or_dtype, device="cuda"):
    """Input dict from ``inputs.make_paged_inputs`` -> dict of device tensors."""
    q_dt = getattr(wl_or_dtype, "q_dtype", wl_or_dtype)
    kv_dt = getattr(wl_or_dtype, "kv_dtype", wl_or_dtype)
    return dict(q=to_device(inp["q"], q_dt, device), k_cache=to_device(inp["k_cache"], kv_dt, device),
                v_cache=to_device(inp["v_cache"], kv_dt, device),
                block_tables=to_device(inp["block_tables"], None, device),
                context_lens=to_device(inp["context_lens"], None, device),
                cu_q_lens=to_device(inp["cu_q_lens"], None, device))


def decode_noalloc(p: Params, q, k_cache, v_cache, block_tables, context_lens, out=None,
                   dev_status=None, stream=None):
    """pa_decode_noalloc: decode with the split partials in the library's
    static device scratch (for callers that cannot allocate at call time).
    Raises PaError(PA_ERR_WORKSPACE) when the partials exceed the scratch."""
    fn = load().pa_decode_noalloc
    if out is None:
        out = _empty_out(q, p)
    _check(fn(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
              _ptr(context_lens), _ptr(out), _ptr(dev_status), _stream(stream)),
           "pa_decode_noalloc")
    return out


# ---- the serving step (include/paged_gqa_serving.h) ---------------------------
# These check what the C entry points cannot see: that each tensor has the
# dtype and the extent that the parameters promise, on one device.

def make_rows(total_rows, max_rows, *, source_rows=0, mask_words=0, q_stride=0, k_stride=0,
              v_stride=0) -> Rows:
    """``pa_rows``: packed rows, their bound per sequence, strides in elements (0: contiguous)."""
    return Rows(total_rows, max_rows, source_rows, mask_words, q_stride, k_stride, v_stride)


def prompt_params(*, num_seqs, num_q_heads, num_kv_heads, head_dim, scale=None, dtype="bf16",
                  out_dtype="f32", debug_timeout=0) -> Params:
    """Params of pa_prompt, which has no pages."""
    return make_params(num_seqs=num_seqs, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
                       head_dim=head_dim, page_size=0, num_pages=0, max_blocks_per_seq=0,
                       max_context_len=0, scale=scale, dtype=dtype, out_dtype=out_dtype,
                       debug_timeout=debug_timeout)


_DTYPES, _I32 = (), None  # torch's dtypes by dtype code, and its int32, once known


def _dtypes():
    global _DTYPES, _I32
    if not _DTYPES:
        import torch
        _DTYPES, _I32 = (torch.float32, torch.float16, torch.bfloat16), torch.int32
    return _DTYPES


def _int32():
    _dtypes()
    return _I32


# The messages are put together only when a check fails, and each property of a
# tensor is asked for once: a small call's kernels take less time than careless
# checks would.

def _ints(t, n, dev, what):
    """Pointer of a contiguous int32 tensor of at least n elements on device number dev."""
    if t.dtype is not (_I32 or _int32()) or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous int32 tensor of at least {n} elements on cuda:{dev}")
    return t.data_ptr()


def _table(t, rows, width, dev, what):
    """Pointer of a contiguous int32 table of ``rows`` rows or more, each ``width`` wide: flat, or with that last dimension."""
    shape = t.shape
    if (t.dtype is not (_I32 or _int32()) or t.get_device() != dev or not t.is_contiguous()
            or (shape[0] < rows or shape[1] != width if len(shape) == 2
                else t.numel() < rows * width or len(shape) > 1 and shape[-1] != width)):
        raise ValueError(f"{what}: a contiguous int32 tensor of at least {rows} rows of {width} elements on cuda:{dev}")
    return t.data_ptr()


def _packed(t, code, rows, heads, dim, stride, dev, what):
    """Pointer of packed rows [rows or more][heads][dim], ``stride`` elements between rows."""
    shape = t.shape
    if (t.get_device() != dev or t.dtype is not _dtypes()[code] or len(shape) != 3 or shape[0] < rows
            or shape[1] != heads or shape[2] != dim
            or not (t.is_contiguous() if stride in (0, heads * dim) else t.stride() == (stride, dim, 1))):
        raise ValueError(f"{what}: [{rows}][{heads}][{dim}] of {_dtypes()[code]}, rows "
                         f"{stride or heads * dim} elements apart, on cuda:{dev}")
    return t.data_ptr()


def _pool(t, p, dev, what):
    """Pointer of a K or V pool: the last slot of the last head and page lies inside the tensor."""
    last = p.num_pages * p.page_size * p.num_kv_heads * p.head_dim
    if p.head_stride or p.token_stride or p.page_stride:
        hs = p.head_stride or p.head_dim
        ts = p.token_stride or p.num_kv_heads * hs
        ps = p.page_stride or p.page_size * ts
        last = (p.num_pages - 1) * ps + (p.page_size - 1) * ts + (p.num_kv_heads - 1) * hs + p.head_dim
    if (t.get_device() != dev or t.dtype is not _dtypes()[p.kv_dtype]
            or (t.numel() < last if t.is_contiguous()
                else not (p.head_stride or p.token_stride or p.page_stride) or _elements_behind(t) < last)):
        raise ValueError(f"{what}: {last} elements of {_dtypes()[p.kv_dtype]} on cuda:{dev}, contiguous unless "
                         "the parameters give strides")
    return t.data_ptr()


def _elements_behind(t):
    """Elements of t's storage from its first one on."""
    return t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()


def _scratch(t, dev):
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on cuda:{dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _status(t, dev):
    return None if t is None else _ints(t, 1, dev, "dev_status")


def _call(name, dev, stream, *args):
    """The entry point with device number dev current, on the given stream or that device's current one."""
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    torch = sys.modules["torch"]  # the tensors came from it, and so CUDA is set up
    if torch._C._cuda_getDevice() != dev:  # torch.cuda.current_device() asks whether it is
        with torch.cuda.device(dev):
            return _call(name, dev, stream, *args)
    # the current stream's handle as torch's own generated launchers get it: torch.cuda.current_stream()
    # builds a Stream object first, which takes longer (2.8 us) than a kernel's launch
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    code = getattr(_lib or load(), name)(*args, handle)
    if code:
        raise PaError(code, name)


def _new(make, size, dtype, like, stream):
    """A tensor made for a call on `stream`: filled there, and not handed out again before the call has run."""
    import torch
    with torch.cuda.stream(stream):  # None: the current one
        return make(size, dtype=dtype, device=like.device)


def _packed_out(p, r, q, out, stream):
    import torch
    if out is None:
        out = _new(torch.zeros, (r.total_rows, p.num_q_heads, p.head_dim), _dtypes()[p.out_dtype], q, stream)
    return out


def prompt(p: Params, r: Rows, q, k, v, cu_lens, out=None, dev_status=None, stream=None):
    """Causal attention over whole packed prompts; q [rows][Hq][D], k and v
    [rows][Hkv][D] -> out [rows][Hq][D] in p.out_dtype.  Rows behind the last
    sequence keep what ``out`` held (zeros when it is made here)."""
    n, d, hq, hkv, dev = r.total_rows, p.head_dim, p.num_q_heads, p.num_kv_heads, q.get_device()
    out = _packed_out(p, r, q, out, stream)
    _call("pa_prompt", dev, stream, p, r,
          _packed(q, p.q_dtype, n, hq, d, r.q_stride, dev, "q"), _packed(k, p.kv_dtype, n, hkv, d, r.k_stride, dev, "k"),
          _packed(v, p.kv_dtype, n, hkv, d, r.v_stride, dev, "v"), _ints(cu_lens, p.num_seqs + 1, dev, "cu_lens"),
          _packed(out, p.out_dtype, n, hq, d, 0, dev, "out"), _status(dev_status, dev))
    return out


def tree_workspace_size(p: Params, r: Rows) -> int:
    return int(load().pa_tree_workspace_size(p, r))


def tree(p: Params, r: Rows, q, k, v, cu_lens, tree_mask, k_cache, v_cache, block_tables,
         context_lens, out=None, workspace=None, dev_status=None, stream=None):
    """Attention of drafted tokens over the paged history and one another:
    packed q, k, v as in ``prompt``, tree_mask [rows][mask_words] int32."""
    n, d, hq, hkv, dev, b = r.total_rows, p.head_dim, p.num_q_heads, p.num_kv_heads, q.get_device(), p.num_seqs
    out = _packed_out(p, r, q, out, stream)
    if workspace is None:
        workspace = _new_scratch(tree_workspace_size(p, r), q, stream)
    words = r.mask_words or (r.max_rows + 31) // 32
    _call("pa_tree", dev, stream, p, r,
          _packed(q, p.q_dtype, n, hq, d, r.q_stride, dev, "q"), _packed(k, p.kv_dtype, n, hkv, d, r.k_stride, dev, "k"),
          _packed(v, p.kv_dtype, n, hkv, d, r.v_stride, dev, "v"), _ints(cu_lens, b + 1, dev, "cu_lens"),
          _table(tree_mask, n, words, dev, "tree_mask"), _pool(k_cache, p, dev, "k_cache"),
          _pool(v_cache, p, dev, "v_cache"), _table(block_tables, b, p.max_blocks_per_seq, dev, "block_tables"),
          _ints(context_lens, b, dev, "context_lens"), _packed(out, p.out_dtype, n, hq, d, 0, dev, "out"),
          *_scratch(workspace, dev), _status(dev_status, dev))
    return out


def store(p: Params, r: Rows, k, v, cu_lens, k_cache, v_cache, block_tables, context_lens,
          row_index=None, dev_status=None, stream=None):
    """Writes packed K/V rows (or, with row_index, chosen rows of them) to
    each sequence's last positions; k_cache and v_cache change in place."""
    n, d, hkv, dev, b = r.total_rows, p.head_dim, p.num_kv_heads, k.get_device(), p.num_seqs
    src = r.source_rows or n
    _call("pa_store", dev, stream, p, r,
          _packed(k, p.kv_dtype, src, hkv, d, r.k_stride, dev, "k"),
          _packed(v, p.kv_dtype, src, hkv, d, r.v_stride, dev, "v"), _ints(cu_lens, b + 1, dev, "cu_lens"),
          None if row_index is None else _ints(row_index, n, dev, "row_index"), _pool(k_cache, p, dev, "k_cache"),
          _pool(v_cache, p, dev, "v_cache"), _table(block_tables, b, p.max_blocks_per_seq, dev, "block_tables"),
          _ints(context_lens, b, dev, "context_lens"), _status(dev_status, dev))


def pages_workspace_size(p: Params) -> int:
    return int(load().pa_pages_workspace_size(p))


def _new_scratch(n, like, stream):
    import torch
    return _new(torch.empty, max(n, 1), torch.uint8, like, stream)


def _bookkeeping(p, refcounts, block_tables, context_lens, dev):
    return (_ints(refcounts, p.num_pages, dev, "refcounts"),
            _table(block_tables, p.num_seqs, p.max_blocks_per_seq, dev, "block_tables"),
            _ints(context_lens, p.num_seqs, dev, "context_lens"))


def pages_resize(p: Params, refcounts, block_tables, context_lens, new_lens, pairs, workspace=None,
                 dev_status=None, stream=None):
    """Reserves, trims and frees pages: sequence s goes to new_lens[s] tokens
    (negative: left alone).  pairs [num_seqs][2] gets the copies to make."""
    dev = refcounts.get_device()
    if workspace is None:
        workspace = _new_scratch(pages_workspace_size(p), refcounts, stream)
    _call("pa_pages_resize", dev, stream, p,
          *_bookkeeping(p, refcounts, block_tables, context_lens, dev), _ints(new_lens, p.num_seqs, dev, "new_lens"),
          _table(pairs, p.num_seqs, 2, dev, "pairs"), *_scratch(workspace, dev), _status(dev_status, dev))


def pages_fork(p: Params, refcounts, block_tables, context_lens, src, dst, dev_status=None, stream=None):
    """Makes each empty sequence dst[i] a copy of src[i] that shares its pages."""
    dev, n = refcounts.get_device(), dst.numel()
    _call("pa_pages_fork", dev, stream, p,
          *_bookkeeping(p, refcounts, block_tables, context_lens, dev), _ints(src, n, dev, "src"),
          _ints(dst, n, dev, "dst"), n, _status(dev_status, dev))


def pages_compact(p: Params, refcounts, block_tables, context_lens, pairs, num_moves, workspace=None,
                  dev_status=None, stream=None):
    """Moves live pages to the low end of the pool, at most len(pairs) of
    them; pairs [n][2] gets the copies to make, num_moves [1] their number."""
    dev, n = refcounts.get_device(), pairs.numel() // 2
    if workspace is None:
        workspace = _new_scratch(pages_workspace_size(p), refcounts, stream)
    _call("pa_pages_compact", dev, stream, p,
          *_bookkeeping(p, refcounts, block_tables, context_lens, dev), _table(pairs, n, 2, dev, "pairs"), n,
          _ints(num_moves, 1, dev, "num_moves"), *_scratch(workspace, dev), _status(dev_status, dev))


def pages_copy(p: Params, k_cache, v_cache, pairs, dev_status=None, stream=None):
    """Copies page pairs[i][0] to pairs[i][1] in one layer's K and V; negative pairs are passed over."""
    dev, n = k_cache.get_device(), pairs.numel() // 2
    _call("pa_pages_copy", dev, stream, p, _pool(k_cache, p, dev, "k_cache"),
          _pool(v_cache, p, dev, "v_cache"), _table(pairs, n, 2, dev, "pairs"), n, _status(dev_status, dev))
