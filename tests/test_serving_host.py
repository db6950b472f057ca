"""The serving-step entry points on the host: struct layouts, the refusals that
come before anything is launched, and a model of how a tree call's work is
shared out.  No test here needs a GPU."""
from __future__ import annotations

import ctypes
import os
import random
import shutil
import subprocess
import tempfile

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
    base = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, num_pages=10,
                max_blocks_per_seq=4, max_context_len=64, dtype="bf16")
    base.update(kw)
    return ops.make_params(**base)


def test_rows_layout_matches_header(lib):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in ops.Rows._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "paged_gqa_serving.h"\nint main(void) {\n'
    src += 'printf("%zu\\n", sizeof(pa_rows));\n' + "".join(f'printf("%zu\\n", offsetof(pa_rows, {n}));\n' for n in names)
    with tempfile.TemporaryDirectory() as d:
        c, x = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src + "return 0; }\n")
        subprocess.run([cc, "-I", os.path.join(ROOT, "include"), c, "-o", x], check=True)
        got = [int(n) for n in subprocess.run([x], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(ops.Rows)] + [getattr(ops.Rows, n).offset for n in names]
    r = ops.make_rows(7, 3, source_rows=9, mask_words=2, q_stride=10, k_stride=20, v_stride=30)
    assert (r.total_rows, r.max_rows, r.source_rows, r.mask_words, r.q_stride, r.k_stride, r.v_stride) == (7, 3, 9, 2, 10, 20, 30)
    lib.pa_rows_init(r)
    assert all(getattr(r, n) == 0 for n in names)


def prompt(lib, p, r, q=BIG, k=BIG, v=BIG, cu=BIG, out=BIG):
    return lib.pa_prompt(p, r, q, k, v, cu, out, None, None)


def tree(lib, p, r, q=BIG, k=BIG, v=BIG, cu=BIG, mask=BIG, kc=BIG, vc=BIG, bt=BIG, cl=BIG, out=BIG, ws=BIG, n=1 << 40):
    return lib.pa_tree(p, r, q, k, v, cu, mask, kc, vc, bt, cl, out, ws, n, None, None)


def store(lib, p, r, k=BIG, v=BIG, cu=BIG, index=None, kc=BIG, vc=BIG, bt=BIG, cl=BIG):
    return lib.pa_store(p, r, k, v, cu, index, kc, vc, bt, cl, None, None)


@pytest.mark.parametrize("call", (prompt, tree))
def test_attention_refusals(lib, call):
    rows = ops.make_rows(5, 3)

    def code(r=rows, **kw):
        return call(lib, params(**kw), r)
    assert call(lib, None, rows) == NULL and call(lib, params(), None) == NULL
    for kw, want in ((dict(num_seqs=0), SHAPE), (dict(num_q_heads=7), SHAPE), (dict(num_q_heads=34), UNSUPPORTED),
                     (dict(head_dim=256), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(scale=0.0), SHAPE),
                     (dict(scale=-0.1), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
                     (dict(kv_dtype="f16"), UNSUPPORTED), (dict(out_dtype="f16"), UNSUPPORTED),
                     (dict(debug_timeout=2), SHAPE)):
        assert code(**kw) == want, kw
    p = params()
    p.q_dtype = 9
    assert call(lib, p, rows) == DTYPE
    for r, want in ((ops.make_rows(-1, 3), SHAPE), (ops.make_rows(5, 0), SHAPE), (ops.make_rows(5, -2), SHAPE),
                    (ops.make_rows(5, 3, q_stride=100), SHAPE), (ops.make_rows(5, 3, k_stride=64), SHAPE),
                    (ops.make_rows(5, 3, v_stride=-128), SHAPE), (ops.make_rows(5, 3, q_stride=515), ALIGN),
                    (ops.make_rows(5, 3, v_stride=129), ALIGN)):
        assert code(r) == want
    for name in ("q", "k", "v", "cu", "out"):
        assert call(lib, params(), rows, **{name: None}) == NULL
        assert call(lib, params(), rows, **{name: ODD}) == ALIGN
    assert code(ops.make_rows(0, 0)) == 0  # nothing to do, nothing launched
    assert call(lib, params(), ops.make_rows(0, 0), q=None) == 0


def test_prompt_ignores_the_page_fields(lib):
    p = ops.prompt_params(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=64, out_dtype="bf16")
    assert prompt(lib, p, ops.make_rows(0, 0)) == 0
    p = ops.prompt_params(num_seqs=60000, num_q_heads=2048, num_kv_heads=2048, head_dim=64)
    assert prompt(lib, p, ops.make_rows(2 ** 31 - 1, 2 ** 31 - 1)) == UNSUPPORTED  # more tiles than 32 bits number


def test_tree_refusals(lib):
    rows = ops.make_rows(5, 3)
    for kw, want in ((dict(page_size=8), UNSUPPORTED), (dict(num_pages=0), SHAPE), (dict(max_blocks_per_seq=0), SHAPE),
                     (dict(num_splits=2), UNSUPPORTED), (dict(sliding_window=5), UNSUPPORTED),
                     (dict(decode_q_rows=2), UNSUPPORTED), (dict(deterministic=3), SHAPE),
                     (dict(strides=(1024, 64, 33)), ALIGN), (dict(strides=(-16, 0, 0)), SHAPE)):
        p = params(max_context_len=1, **kw)
        assert tree(lib, p, rows) == want, kw
        assert ops.tree_workspace_size(p, rows) == 0
    for name in ("mask", "kc", "vc", "bt", "cl", "ws"):
        assert tree(lib, params(), rows, **{name: None}) == NULL
        assert tree(lib, params(), rows, **{name: ODD}) == ALIGN
    assert tree(lib, params(), rows, ws=ctypes.c_void_p((1 << 20) + 16)) == ALIGN
    n = ops.tree_workspace_size(params(), rows)
    assert n > 0 and tree(lib, params(), rows, n=n - 1) == WORKSPACE
    assert tree(lib, params(), ops.make_rows(2000, 1025)) == UNSUPPORTED
    assert tree(lib, params(), ops.make_rows(100, 33, mask_words=1)) == SHAPE
    assert tree(lib, params(), ops.make_rows(5, 3, mask_words=-1)) == SHAPE


def test_store_refusals(lib):
    rows = ops.make_rows(5, 3)
    assert store(lib, None, rows) == NULL and store(lib, params(), None) == NULL
    for name in ("k", "v", "cu", "kc", "vc", "bt", "cl"):
        assert store(lib, params(), rows, **{name: None}) == NULL
        assert store(lib, params(), rows, **{name: ODD}) == ALIGN
    assert store(lib, params(), rows, index=ODD) == ALIGN
    assert store(lib, params(head_dim=80), rows) == UNSUPPORTED
    assert store(lib, params(page_size=64), rows) == UNSUPPORTED
    assert store(lib, params(), ops.make_rows(5, 3, source_rows=4)) == SHAPE  # without an index
    assert store(lib, params(), ops.make_rows(5, 3, k_stride=100)) == SHAPE
    assert store(lib, params(), ops.make_rows(0, 0), k=None) == 0


def test_pages_refusals(lib):
    p = params()
    n = ops.pages_workspace_size(p)
    assert n > 0 and n % 256 == 0
    assert ops.pages_workspace_size(params(num_pages=(1 << 23) + 1)) == 0

    def resize(p=p, ref=BIG, bt=BIG, cl=BIG, new=BIG, pairs=BIG, ws=BIG, n=n):
        return lib.pa_pages_resize(p, ref, bt, cl, new, pairs, ws, n, None, None)

    def fork(p=p, ref=BIG, bt=BIG, cl=BIG, src=BIG, dst=BIG, count=1):
        return lib.pa_pages_fork(p, ref, bt, cl, src, dst, count, None, None)

    def compact(p=p, ref=BIG, bt=BIG, cl=BIG, pairs=BIG, most=4, num=BIG, ws=BIG, n=n):
        return lib.pa_pages_compact(p, ref, bt, cl, pairs, most, num, ws, n, None, None)

    def copy(p=p, kc=BIG, vc=BIG, pairs=BIG, count=1):
        return lib.pa_pages_copy(p, kc, vc, pairs, count, None, None)
    for call, names in ((resize, ("ref", "bt", "cl", "new", "pairs", "ws")), (fork, ("ref", "bt", "cl", "src", "dst")),
                        (compact, ("ref", "bt", "cl", "pairs", "num", "ws")), (copy, ("kc", "vc", "pairs"))):
        assert call(p=None) == NULL
        for name in names:
            assert call(**{name: None}) == NULL, name
            assert call(**{name: ODD}) == ALIGN, name
        for kw, want in ((dict(num_seqs=0), SHAPE), (dict(num_seqs=70000), SHAPE), (dict(page_size=24), UNSUPPORTED),
                         (dict(num_pages=0), SHAPE)):
            assert call(p=params(**kw)) == want, (call, kw)
    assert resize(n=n - 1) == WORKSPACE and compact(n=n - 1) == WORKSPACE
    assert resize(pairs=ctypes.c_void_p((1 << 20) + 4)) == ALIGN
    assert fork(count=-1) == SHAPE and fork(count=0, src=None) == 0
    assert compact(most=-1) == SHAPE
    assert copy(count=-1) == SHAPE and copy(count=0, pairs=None) == 0


# ---- how a tree call's work is shared out ------------------------------------------

def up(a, b):
    return -(-a // b)


def shares(lens, drafts, hkv, tu, tile, kb, start, least, ctas):
    """The pieces that each CTA takes, {unit: [(cta, first block, end, slot, last cta)]}, as the kernels walk them."""
    seqs = []
    for L, T in zip(lens, drafts):
        blocks, width = up(L, kb) + up(T, kb), 2 if T > tile else 1
        seqs.append((up(T, tu), blocks, width, start + width * blocks if T else 0))
    total = sum(hkv * u * c for u, _, _, c in seqs)
    if not total:
        return {}, seqs
    n = min(ctas, max(1, total // least))
    got = {}
    for cta in range(n):
        at, end, s, seq_at = up(total * cta, n), up(total * (cta + 1), n), 0, 0
        while at < end:
            while at >= seq_at + hkv * seqs[s][0] * seqs[s][3]:
                seq_at += hkv * seqs[s][0] * seqs[s][3]
                s += 1
            u, blocks, width, cost = seqs[s]
            unit, o = divmod(at - seq_at, cost)
            take = min(cost - o, end - at)
            at += take
            b0, b1 = (max(x - start + width - 1, 0) // width for x in (o, o + take))
            if b0 < b1:
                whole = b0 == 0 and b1 == blocks
                last = (seq_at + unit * cost + start + width * (blocks - 1)) * n // total
                got.setdefault((s, unit), []).append((cta, b0, b1, -1 if whole else 2 * cta + (b0 == 0), last))
    return got, seqs


@pytest.mark.parametrize("seed", range(40))
def test_shares_cover_every_block_once(seed):
    rng = random.Random(seed)
    n = rng.choice([1, 2, 7, 40])
    lens = [rng.choice([0, 1, rng.randint(0, 300), rng.randint(0, 20000)]) for _ in range(n)]
    drafts = [rng.choice([0, 1, rng.randint(0, 64), rng.randint(0, 300)]) for _ in range(n)]
    hkv, ctas = rng.choice([1, 2, 8]), rng.choice([1, 13, 152])
    if seed % 2:  # two row tiles a unit, blocks of a second one count double
        tile = rng.choice([8, 32, 128])
        tu, kb, start, least = 2 * tile, 128, 5, 2
    else:
        tu, kb, start, least, tile = rng.choice([4, 16, 64]), 64, 1, 1, 1 << 30
    got, seqs = shares(lens, drafts, hkv, tu, tile, kb, start, least, ctas)
    for s, (u, blocks, _, _) in enumerate(seqs):
        for unit in range(hkv * u):
            pieces = got.pop((s, unit))
            assert [x for _, a, b, _, _ in pieces for x in range(a, b)] == list(range(blocks))
            first, last = pieces[0], pieces[-1]
            # the join reads one slot of each CTA from the first to `last`
            assert first[4] == last[0] and [p[0] for p in pieces] == list(range(first[0], last[0] + 1))
            if len(pieces) == 1:
                assert first[3] == -1
            else:
                assert [p[3] for p in pieces] == [2 * first[0] + 1] + [2 * p[0] for p in pieces[1:]]
    assert not got


def test_shares_slots_are_their_own():
    got, _ = shares([700, 5000, 0, 33], [64, 7, 1, 200], 4, 64, 32, 128, 5, 2, 152)
    slots = [p[3] for v in got.values() for p in v if p[3] >= 0]
    assert len(slots) == len(set(slots)) and max(slots) < 2 * 152
    begins = [p[0] for v in got.values() for p in v if p[3] >= 0 and p[3] & 1]
    assert len(begins) == len(set(begins))  # one unit to join begins in a CTA's share


def test_python_checks_see_what_the_library_cannot():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        ops._packed(x, ops.PA_BF16, 4, 2, 64, 0, 0, "q")
    dev = x.get_device()
    assert ops._packed(x, ops.PA_BF16, 4, 2, 64, 0, dev, "q") == x.data_ptr()
    wide = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    assert ops._packed(wide[:, 2:4], ops.PA_BF16, 4, 2, 64, 384, dev, "k") == wide.data_ptr() + 256
    for args in ((x, ops.PA_F16, 4, 2, 64, 0), (x, ops.PA_BF16, 5, 2, 64, 0), (x, ops.PA_BF16, 4, 1, 64, 0),
                 (x, ops.PA_BF16, 4, 2, 128, 0), (x[:, :, :32], ops.PA_BF16, 4, 2, 32, 0),
                 (wide[:, 2:4], ops.PA_BF16, 4, 2, 64, 0), (x, ops.PA_BF16, 4, 2, 64, 384)):
        with pytest.raises(ValueError):
            ops._packed(*args, dev, "q")
    i = torch.zeros(6, dtype=torch.int32)
    assert ops._ints(i, 6, dev, "i") == i.data_ptr()
    for t, n in ((i, 7), (i.long(), 6), (i.float(), 6), (torch.zeros(12, dtype=torch.int32)[::2], 6)):
        with pytest.raises(ValueError):
            ops._ints(t, n, dev, "i")
    p = params(num_pages=3)
    pool = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    assert ops._pool(pool, p, dev, "k") == pool.data_ptr()
    with pytest.raises(ValueError):
        ops._pool(pool[:2], p, dev, "k")
    layers = torch.zeros(3, 2, 16, 2, 64, dtype=torch.bfloat16)  # two layers' pages side by side
    with pytest.raises(ValueError):
        ops._pool(layers[:, 1], p, dev, "k")
    assert ops._pool(layers[:, 1], params(num_pages=3, strides=(2 * 16 * 128, 128, 64)), dev, "k")
    head_major = params(num_pages=3, strides=(2 * 16 * 64, 64, 16 * 64))
    assert ops._pool(torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16), head_major, dev, "k")
    with pytest.raises(ValueError):
        ops._pool(pool, params(num_pages=3, strides=(4096, 256, 64)), dev, "k")
