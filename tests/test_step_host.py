"""pa_rotate, pa_verify, pa_key_weights and pa_evict on the host: the struct's
layout and the refusals that come before anything is launched.  No test here
needs a GPU."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from paged_kv_gqa_02_gb300 import build, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = ctypes.c_void_p(1 << 20)       # aligned, never dereferenced: every call below is refused
ODD = ctypes.c_void_p((1 << 20) + 2)
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 5, 6


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.load()


def params(**kw):
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, num_pages=10, max_blocks_per_seq=4,
                max_context_len=64, dtype="bf16")
    base.update(kw)
    return ops.make_params(**base)


def test_rope_layout_matches_header(lib, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in ops.Rope._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "paged_gqa_serving.h"\nint main(void) {\nprintf("%zu\\n", sizeof(pa_rope));\n'
    src += "".join(f'printf("%zu\\n", offsetof(pa_rope, {n}));\n' for n in names) + "return 0; }\n"
    (tmp_path / "l.c").write_text(src)
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = [int(n) for n in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(ops.Rope)] + [getattr(ops.Rope, n).offset for n in names]
    t = ops.make_rope(64, table_rows=9, interleaved=True, eps=0.5, sections=(1, 2, 3), q_out_stride=4, k_out_stride=5)
    assert (t.rotary_dim, t.interleaved, t.axes, list(t.sections), t.table_rows, t.eps) == (64, 1, 3, [1, 2, 3], 9, 0.5)
    lib.pa_rope_init(t)
    assert (t.rotary_dim, t.interleaved, t.axes, list(t.sections), t.table_rows, t.q_out_stride, t.k_out_stride) == (0, 0, 0, [0, 0, 0], 0, 0, 0)
    assert abs(t.eps - 1e-6) < 1e-12


def rotate(lib, p=None, r=None, t=None, **kw):
    a = dict(q=BIG, k=BIG, v=BIG, cu=BIG, table=BIG, pos=None, cl=BIG, qw=None, kw=None, qo=ctypes.c_void_p(1 << 21), ko=ctypes.c_void_p(1 << 22),
             kc=BIG, vc=BIG, bt=BIG)
    a.update(kw)
    return lib.pa_rotate(p or params(), r or ops.make_rows(5, 3), t or ops.make_rope(64, table_rows=9), *a.values(), None, None)


def test_rotate_refuses(lib):
    assert lib.pa_rotate(None, None, None, *[None] * 14, None, None) == NULL
    for name in ("q", "k", "v", "cu", "table", "cl", "qo", "vc", "bt"):
        assert rotate(lib, **{name: None}) == NULL, name
    assert rotate(lib, kc=None, ko=None) == NULL
    assert rotate(lib, kc=None, cl=None) == NULL
    for name in ("q", "k", "v", "cu", "table", "pos", "cl", "qw", "kw", "qo", "ko", "kc", "vc", "bt"):
        assert rotate(lib, **{name: ODD}) == ALIGN, name
    for rope in (ops.make_rope(24, table_rows=9), ops.make_rope(80, table_rows=9), ops.make_rope(-16, table_rows=9), ops.make_rope(64),
                 ops.make_rope(64, table_rows=9, sections=(16, 17)), ops.make_rope(64, table_rows=9, sections=(-1, 33)),
                 ops.make_rope(64, table_rows=9, eps=-1.0), ops.make_rope(64, table_rows=9, eps=float("nan")),
                 ops.make_rope(64, table_rows=9, q_out_stride=64), ops.make_rope(64, table_rows=9, k_out_stride=64)):
        assert rotate(lib, t=rope) == SHAPE
    wrong = ops.make_rope(64, table_rows=9)
    wrong.sections[0] = 32
    assert rotate(lib, t=wrong) == SHAPE
    wrong = ops.make_rope(64, table_rows=9)
    wrong.axes = 4
    assert rotate(lib, t=wrong) == SHAPE
    assert rotate(lib, t=ops.make_rope(64, table_rows=9, q_out_stride=8 * 64 + 4)) == ALIGN
    assert rotate(lib, p=params(head_dim=96)) == UNSUPPORTED
    assert rotate(lib, p=params(page_size=8)) == UNSUPPORTED
    assert rotate(lib, p=params(dtype="bf16", kv_dtype="f16")) == UNSUPPORTED
    assert rotate(lib, p=params(num_seqs=0)) == SHAPE
    assert rotate(lib, r=ops.make_rows(5, 0)) == SHAPE
    assert rotate(lib, r=ops.make_rows(1 << 30 | 1, 3)) == UNSUPPORTED
    # rows over their input with another stride
    assert rotate(lib, qo=BIG, r=ops.make_rows(5, 3, q_stride=640)) == SHAPE
    assert rotate(lib, ko=BIG, r=ops.make_rows(5, 3, k_stride=640)) == SHAPE
    assert rotate(lib, r=ops.make_rows(0, 0)) == 0


def verify(lib, p=None, r=None, vocab=100, **kw):
    a = dict(logits=BIG, draft=BIG, tokens=BIG, parents=BIG, cu=BIG, heat=BIG, uniform=BIG, noise=BIG, cl=BIG, acc=BIG, ends=BIG, nexts=BIG, lens=BIG)
    a.update(kw)
    return lib.pa_verify(p or ops.verify_params(num_seqs=2), r or ops.make_rows(5, 3), vocab, *a.values(), None, None)


def test_verify_refuses(lib):
    assert lib.pa_verify(None, None, 1, *[None] * 13, None, None) == NULL
    for name in ("logits", "tokens", "parents", "cu", "heat", "uniform", "noise", "acc", "ends", "nexts", "cl", "lens"):
        assert verify(lib, **{name: None}) == NULL, name
    for name in ("logits", "draft"):
        assert verify(lib, **{name: ctypes.c_void_p((1 << 20) + 1)}) == ALIGN
    for name in ("tokens", "parents", "cu", "heat", "uniform", "noise", "cl", "acc", "ends", "nexts", "lens"):
        assert verify(lib, **{name: ODD}) == ALIGN, name
    assert verify(lib, vocab=0) == SHAPE
    assert verify(lib, vocab=(1 << 28) + 1) == UNSUPPORTED
    assert verify(lib, r=ops.make_rows(5, 3, q_stride=99)) == SHAPE
    assert verify(lib, r=ops.make_rows(5, 3, k_stride=99)) == SHAPE
    assert verify(lib, r=ops.make_rows(2000, 1025)) == UNSUPPORTED
    assert verify(lib, r=ops.make_rows(-1, 3)) == SHAPE
    assert verify(lib, p=ops.verify_params(num_seqs=0)) == SHAPE


def key_weights(lib, p=None, r=None, decay=1.0, n=1 << 40, **kw):
    a = dict(q=BIG, cu=BIG, kc=BIG, bt=BIG, cl=BIG)
    b = dict(weights=BIG, ws=BIG)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    return lib.pa_key_weights(p or params(), r or ops.make_rows(5, 3), *a.values(), decay, *b.values(), n, None, None)


def test_key_weights_refuses(lib):
    for name in ("q", "cu", "kc", "bt", "cl", "weights", "ws"):
        assert key_weights(lib, **{name: None}) == NULL, name
        assert key_weights(lib, **{name: ODD}) == ALIGN, name
    for decay in (-0.1, 1.5, float("nan")):
        assert key_weights(lib, decay=decay) == SHAPE
    need = ops.key_weights_workspace_size(params(), ops.make_rows(5, 3))
    assert need > 0 and key_weights(lib, n=need - 1) == WORKSPACE
    for bad, code in ((dict(head_dim=256), UNSUPPORTED), (dict(num_q_heads=34), UNSUPPORTED), (dict(num_q_heads=7), SHAPE), (dict(scale=0.0), SHAPE),
                      (dict(scale=float("inf")), SHAPE), (dict(sliding_window=5), UNSUPPORTED), (dict(num_splits=2), UNSUPPORTED),
                      (dict(decode_q_rows=2), UNSUPPORTED), (dict(page_size=64), UNSUPPORTED), (dict(max_context_len=-1), SHAPE),
                      (dict(kv_dtype="f32"), UNSUPPORTED), (dict(deterministic=2), SHAPE)):
        assert key_weights(lib, p=params(**bad)) == code, bad
        assert ops.key_weights_workspace_size(params(**bad), ops.make_rows(5, 3)) == 0
    assert key_weights(lib, r=ops.make_rows(5, 3, q_stride=500)) == SHAPE
    assert key_weights(lib, r=ops.make_rows(5, 3, q_stride=516)) == ALIGN
    assert key_weights(lib, r=ops.make_rows(0, 0)) == 0


def test_key_weights_refuses_more_than_it_can_count(lib):
    big = dict(num_seqs=65535, num_kv_heads=65535, num_q_heads=65535, max_blocks_per_seq=1 << 27, max_context_len=0)
    for bad, r in ((big, ops.make_rows(5, 3)), (dict(big, num_q_heads=16 * 4096, num_kv_heads=4096), ops.make_rows(5, 1)),
                   (dict(max_blocks_per_seq=1 << 27, max_context_len=0), ops.make_rows(1 << 20, 1 << 20))):
        assert key_weights(lib, p=params(**bad), r=r) == UNSUPPORTED, bad
        assert ops.key_weights_workspace_size(params(**bad), r) == 0
    # the longest table of one sequence: its scores and pieces count in 64 bits
    p, r = params(num_seqs=1, num_q_heads=1, num_kv_heads=1, max_blocks_per_seq=1 << 26, max_context_len=0), ops.make_rows(1, 1)
    assert ops.key_weights_workspace_size(p, r) >= 8 * p.page_size << 26


def evict(lib, p=None, first=0, recent=0, **kw):
    a = dict(kc=BIG, vc=BIG, bt=BIG, cl=BIG, ref=BIG, w=BIG, keep=BIG)
    b = dict(out=ctypes.c_void_p(1 << 21), kept=BIG, lens=BIG)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    return lib.pa_evict(p or params(), *a.values(), first, recent, *b.values(), None, None)


def test_evict_refuses(lib):
    for name in ("kc", "vc", "bt", "cl", "w", "keep", "out", "kept", "lens"):
        assert evict(lib, **{name: None}) == NULL, name
    for name in ("kc", "vc", "bt", "cl", "ref", "w", "keep", "out", "kept", "lens"):
        assert evict(lib, **{name: ODD}) == ALIGN, name
    assert evict(lib, first=-1) == SHAPE and evict(lib, recent=-1) == SHAPE
    assert evict(lib, out=BIG) == SHAPE
    assert evict(lib, p=params(max_blocks_per_seq=1 << 20)) == UNSUPPORTED
    assert evict(lib, p=params(num_seqs=65535, num_kv_heads=65535, num_q_heads=65535)) == UNSUPPORTED
    assert evict(lib, p=params(num_seqs=65535, num_kv_heads=129, num_q_heads=129)) == UNSUPPORTED
    assert evict(lib, p=params(head_dim=32)) == UNSUPPORTED
    assert evict(lib, p=params(strides=(0, 4, 0))) == ALIGN


# ---- the Python calls' own checks --------------------------------------------------

torch = pytest.importorskip("torch")


class Passed(Exception):
    """Every check of the arguments passed."""


@pytest.fixture
def on_the_host(lib, monkeypatch):
    """Tensors of the CPU (device -1) go through the checks; nothing is called."""
    def call(name, dev, stream, *args):
        raise Passed(name)
    monkeypatch.setattr(ops, "_call", call)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f32(*shape):
    return torch.zeros(shape)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def rotate_call(**kw):
    a = dict(q=bf16(5, 8, 64), k=bf16(5, 2, 64), cu_lens=i32(3), table=f32(9, 64), v=bf16(5, 2, 64), positions=i32(1, 5), context_lens=i32(2),
             q_weight=bf16(64), k_weight=bf16(64), q_out=bf16(5, 8, 64), k_out=bf16(5, 2, 64), k_cache=bf16(10, 16, 2, 64), v_cache=bf16(10, 16, 2, 64),
             block_tables=i32(2, 4))
    a.update(kw)
    q, k, starts, table = (a.pop(x) for x in ("q", "k", "cu_lens", "table"))
    return ops.rotate(params(), ops.make_rows(5, 3), ops.make_rope(64, table_rows=9), q, k, starts, table, **a)


def verify_call(**kw):
    a = dict(logits=bf16(5, 100), draft_logits=bf16(5, 100), tokens=i32(5), parents=i32(5), cu_lens=i32(3), temperature=f32(2), uniform=f32(5),
             noise=f32(2, 100), context_lens=i32(2), accepted=i32(5), accepted_cu=i32(3), next_tokens=i32(2), new_lens=i32(2))
    a.update(kw)
    return ops.verify(ops.verify_params(num_seqs=2), ops.make_rows(5, 3), *a.values())


def key_weights_call(**kw):
    a = dict(q=bf16(5, 8, 64), cu_lens=i32(3), k_cache=bf16(10, 16, 2, 64), block_tables=i32(2, 4), context_lens=i32(2), weights=f32(2, 2, 64))
    a.update(kw)
    return ops.key_weights(params(), ops.make_rows(5, 3), *a.values(), workspace=torch.zeros(1, dtype=torch.uint8))


def evict_call(**kw):
    a = dict(k_cache=bf16(10, 16, 2, 64), v_cache=bf16(10, 16, 2, 64), block_tables=i32(2, 4), context_lens=i32(2), weights=f32(2, 2, 64),
             keep_lens=i32(2), weights_out=f32(2, 2, 64), kept=i32(2, 2, 64), new_lens=i32(2))
    a.update(kw)
    ref = a.pop("refcounts", i32(10))
    return ops.evict(params(), *a.values(), refcounts=ref)


WRONG = [
    (rotate_call, dict(q=[bf16(5, 8, 32), bf16(4, 8, 64), f32(5, 8, 64), bf16(5, 64, 8).transpose(1, 2)], k=[bf16(5, 3, 64)], cu_lens=[i32(2), f32(3)],
                       table=[f32(8, 64), bf16(9, 64)], v=[bf16(5, 1, 64)], positions=[i32(2, 4), i32(1, 4), i32(5, 1)], context_lens=[i32(1)],
                       q_weight=[bf16(32), f32(64)], k_weight=[bf16(128)], q_out=[bf16(5, 2, 64)], k_out=[f32(5, 2, 64)],
                       k_cache=[bf16(9, 16, 2, 64)], v_cache=[f32(10, 16, 2, 64)], block_tables=[i32(2, 5), i32(1, 4)])),
    (verify_call, dict(logits=[bf16(4, 100), f32(5, 100), bf16(5, 100, 1), bf16(100, 5).T], draft_logits=[bf16(5, 99), bf16(4, 100)], tokens=[i32(4)],
                       parents=[f32(5)], cu_lens=[i32(2)], temperature=[f32(1), i32(2)], uniform=[f32(4)], noise=[f32(2, 99), bf16(2, 100)],
                       context_lens=[i32(1)], accepted=[i32(4)], accepted_cu=[i32(2)], next_tokens=[i32(1)], new_lens=[i32(1)])),
    (key_weights_call, dict(q=[bf16(5, 4, 64)], cu_lens=[i32(2)], k_cache=[bf16(10, 16, 64)], block_tables=[i32(2, 3)], context_lens=[i32(1)],
                            weights=[f32(2, 2, 63), f32(2, 1, 64), f32(1, 2, 64), bf16(2, 2, 64), f32(2, 128), f32(2, 64, 2).transpose(1, 2)])),
    (evict_call, dict(k_cache=[bf16(9, 16, 2, 64)], v_cache=[f32(10, 16, 2, 64)], block_tables=[i32(2, 5)], context_lens=[i32(1)], keep_lens=[i32(1)],
                      weights=[f32(2, 2, 65), i32(2, 2, 64)], weights_out=[f32(1, 2, 64)], kept=[f32(2, 2, 64), i32(2, 2, 60)], new_lens=[i32(1)],
                      refcounts=[i32(9)])),
]


def test_the_right_tensors_pass(on_the_host):
    for call, _ in WRONG:
        with pytest.raises(Passed):
            call()
    for call, kw in ((rotate_call, dict(v=None, k_cache=None, v_cache=None, block_tables=None)), (rotate_call, dict(positions=None, q_weight=None)),
                     (verify_call, dict(draft_logits=None)), (verify_call, dict(context_lens=None, new_lens=None)), (evict_call, dict(refcounts=None)),
                     (rotate_call, dict(positions=i32(5))), (verify_call, dict(logits=bf16(7, 100)))):
        with pytest.raises(Passed):
            call(**kw)


@pytest.mark.parametrize("call,name,i", [(call, name, i) for call, by in WRONG for name, bad in by.items() for i in range(len(bad))])
def test_other_tensors_are_refused(on_the_host, call, name, i):
    bad = dict((c, by) for c, by in WRONG)[call][name][i]
    with pytest.raises(ValueError):
        call(**{name: bad})
