"""Prompt and tree attention on the GPU against plain 64-bit forms
(serving_ref): element by element, within bounds derived there."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gqa_02_gb300 import build, ops
import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.load()


def packed(total, hq, hkv, d, dtype, seed, fused=False):
    """q, k, v of packed rows; fused: slices of one [rows][Hq + 2 Hkv][D] projection."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((total, hq + 2 * hkv, d), generator=gen).to(ref.DT[dtype]).cuda()
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return parts if fused else tuple(t.contiguous() for t in parts)


def strides_of(fused, hq, hkv, d):
    n = (hq + 2 * hkv) * d
    return dict(q_stride=n, k_stride=n, v_stride=n) if fused else {}


TYPES = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


def run_prompt(lens, dtype, out_dtype, hq, hkv, d, seed=1, pad=0, fused=False, scale=None):
    total = sum(lens) + pad
    q, k, v = packed(total, hq, hkv, d, dtype, seed, fused)
    p = ops.prompt_params(num_seqs=len(lens), num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=dtype,
                          out_dtype=out_dtype, scale=scale)
    r = ops.make_rows(total, max(lens), **strides_of(fused, hq, hkv, d))
    out = torch.full((total, hq, d), 7.0, dtype=ref.DT[out_dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.prompt(p, r, q, k, v, ref.cu(lens), out=out, dev_status=status)
    assert int(status.item()) == 0
    want, tol = ref.prompt_ref(q, k, v, lens, p.scale, dtype, out_dtype)
    n = sum(lens)
    ref.assert_close(out[:n], want[:n], tol[:n], f"{lens} {dtype}")
    assert (out[n:] == 7.0).all(), "rows behind the last sequence were written"
    return q, k, v, out


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("d", (64, 128))
def test_prompt_lengths(dtype, out_dtype, d):
    run_prompt([1, 0, 5, 31, 127, 128, 129, 300], dtype, out_dtype, 8, 2, d, pad=3)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (6, 2), (10, 2), (7, 1), (16, 2), (16, 1)])
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_prompt_head_groups(dtype, hq, hkv):
    run_prompt([257, 40, 512], dtype, dtype, hq, hkv, 128, seed=hq)


@pytest.mark.parametrize("dtype", ("f32", "f16"))
def test_prompt_slices_of_a_projection(dtype):
    run_prompt([100, 1, 260], dtype, dtype, 8, 4, 64, pad=2, fused=True)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_prompt_large_scores(dtype, out_dtype):
    """Scores in the tens: the running max moves, weights are peaked."""
    run_prompt([700], dtype, out_dtype, 4, 1, 128, scale=1.0)


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
def test_prompt_more_items_than_ctas(dtype):
    run_prompt([900, 3, 1500, 64, 1, 1200], dtype, dtype, 16, 8, 64, pad=1)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("value", (float("nan"), float("inf"), -float("inf")))
def test_prompt_bad_values_reach_only_later_rows(dtype, out_dtype, value):
    """A NaN or infinity in K or V of token j leaves rows before j as they were, bit for bit."""
    lens, hq, hkv, d = [330, 90], 4, 2, 64
    q, k, v, clean = run_prompt(lens, dtype, out_dtype, hq, hkv, d)
    p = ops.prompt_params(num_seqs=2, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=dtype, out_dtype=out_dtype)
    for j, into in ((200, v), (129, v), (33, v), (200, k)):
        kept = into[j, 1].clone()
        into[j, 1, 5] = value
        out = ops.prompt(p, ops.make_rows(420, 330), q, k, v, ref.cu(lens))
        assert torch.equal(out[:j], clean[:j]) and torch.equal(out[330:], clean[330:])
        assert torch.equal(out[j:330, :2], clean[j:330, :2])  # the other kv head's rows
        if into is v:
            seen = out[j:330, 2:, 5]
            assert (seen.isnan() if math.isnan(value) else seen == value).all()
            other = [c for c in range(d) if c != 5]
            if out_dtype != "f32":  # the rest of the row is what it was
                assert torch.equal(out[j:330, 2:, other], clean[j:330, 2:, other])
        into[j, 1] = kept


def test_prompt_repeats_bit_for_bit_and_replays():
    lens = [500, 20, 333]
    q, k, v, first = run_prompt(lens, "bf16", "bf16", 16, 4, 128)
    p = ops.prompt_params(num_seqs=3, num_q_heads=16, num_kv_heads=4, head_dim=128, dtype="bf16", out_dtype="bf16")
    r, c = ops.make_rows(853, 500), ref.cu(lens)
    out = torch.zeros_like(first)
    graph = torch.cuda.CUDAGraph()
    ops.prompt(p, r, q, k, v, c, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    with torch.cuda.graph(graph):
        ops.prompt(p, r, q, k, v, c, out=out)
    c.copy_(ref.cu([20, 500, 333]))  # other lengths, the same capture
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, tol = ref.prompt_ref(q, k, v, [20, 500, 333], p.scale, "bf16", "bf16")
        ref.assert_close(out, want, tol)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_prompt_refused_rows_are_left(dtype):
    """Ends outside the rows, descending ends, a sequence over max_rows: flagged, skipped."""
    q, k, v = packed(100, 4, 2, 64, dtype, 3)
    p = ops.prompt_params(num_seqs=3, num_q_heads=4, num_kv_heads=2, head_dim=64, dtype=dtype, out_dtype=dtype)
    for ends, good in (([0, 40, 30, 60], (0, 30)),  # rows 30..39 are two sequences'
                        ([0, 20, 40, 200], (20, 40)), ([0, 10, 90, 100], (90, 100)),
                       ([-5, 10, 20, 30], (20, 30))):
        out = torch.full_like(q, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.prompt(p, ops.make_rows(100, 50), q, k, v, torch.tensor(ends, dtype=torch.int32, device="cuda"), out=out,
                   dev_status=status)
        assert int(status.item()) == ops.PA_DEV_BAD_LEN
        a, b = good
        want, tol = ref.prompt_ref(q[a:b], k[a:b], v[a:b], [b - a], p.scale, dtype, dtype)
        ref.assert_close(out[a:b], want, tol)
    assert (out[30:] == 7.0).all() and (out[:10] == 7.0).all()


def run_tree(lens, drafts, dtype, out_dtype, hq, hkv, d, page, seed=1, empty=0.0, words=0, fused=False,
             head_major=False, mask=None, pad=0, **kw):
    gen = torch.Generator().manual_seed(seed)
    pool = ref.Pool(lens, page, hkv, d, dtype, gen, head_major=head_major)
    total = sum(drafts)
    q, k, v = packed(total + pad, hq, hkv, d, dtype, seed + 50, fused)
    n_words = words or -(-max(drafts) // 32)
    if mask is None:
        mask = ref.random_mask(list(drafts) + [1] * pad, n_words, gen, empty)
    p = pool.params(hq, out_dtype=out_dtype, **kw)
    r = ops.make_rows(total + pad, max(drafts), mask_words=words, **strides_of(fused, hq, hkv, d))
    out = torch.full((total + pad, hq, d), 7.0, dtype=ref.DT[out_dtype], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = ref.cu(drafts)
    ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, out=out, dev_status=status)
    assert int(status.item()) == 0
    want, tol = ref.tree_ref(q[:total], k[:total], v[:total], drafts, mask, *pool.kv, pool.tables, lens, p.scale,
                             dtype, out_dtype)
    ref.assert_close(out[:total], want, tol, f"{lens} {drafts} {dtype}")
    assert (out[total:] == 7.0).all()
    return pool, p, r, q, k, v, c, mask, out


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_tree_lengths(dtype, out_dtype, d, page):
    run_tree([0, 1, 31, 32, 33, 128, 129, 700, 0], [5, 1, 0, 16, 7, 33, 64, 26, 1], dtype, out_dtype, 8, 2, d, page)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (10, 2), (14, 2), (16, 2), (16, 1)])
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_tree_head_groups(dtype, hq, hkv):
    run_tree([300, 77], [40, 9], dtype, dtype, hq, hkv, 128, 16, seed=hq)


@pytest.mark.parametrize("dtype", ("f32", "f16"))
def test_tree_one_long_history_over_all_shares(dtype):
    run_tree([5000], [3], dtype, dtype, 4, 1, 64, 32)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_tree_many_drafts(dtype, out_dtype):
    """More drafts than a key tile and than a unit, mask rows wider than needed."""
    run_tree([100, 0, 260], [150, 200, 129], dtype, out_dtype, 8, 4, 64, 16, words=9, pad=2)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_tree_rows_that_see_nothing(dtype):
    *_, out = run_tree([0, 0, 50], [40, 7, 9], dtype, dtype, 8, 2, 128, 32, empty=0.5)
    _, _, _, _, _, _, _, mask, out = run_tree([0], [33], dtype, dtype, 4, 2, 64, 16,
                                              mask=torch.zeros(33, 2, dtype=torch.int32, device="cuda"))
    assert (out == 0).all()


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_tree_strides(dtype):
    run_tree([70, 200], [9, 20], dtype, dtype, 8, 4, 128, 16, fused=True, head_major=True, pad=1)


@pytest.mark.parametrize("dtype", ("f32", "f16"))
def test_tree_many_sequences(dtype):
    n = 70
    run_tree([(i * 37) % 90 for i in range(n)], [(i * 5) % 7 for i in range(n)], dtype, dtype, 4, 2, 64, 16)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("value", (float("nan"), float("inf")))
def test_tree_bad_values_reach_only_rows_that_see_them(dtype, out_dtype, value):
    pool, p, r, q, k, v, c, mask, clean = run_tree([200, 40], [40, 6], dtype, out_dtype, 4, 2, 64, 16)
    see = ref.bits(mask, 0, 40)
    for j, into in ((7, v), (33, v), (12, k)):
        kept = into[j].clone()
        into[j, 0, 3] = value
        out = ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context)
        blind = torch.nonzero(~see[:, j]).flatten()
        assert torch.equal(out[blind], clean[blind]) and torch.equal(out[40:], clean[40:])
        if into is v:
            seen = out[:40][see[:, j]][:, :2, 3]
            assert (seen.isnan() if math.isnan(value) else seen == value).all()
        into[j] = kept


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_tree_pages_outside_the_pool_and_bad_lengths(dtype):
    gen = torch.Generator().manual_seed(4)
    lens, drafts = [300, 90, 150], [10, 4, 7]
    pool = ref.Pool(lens, 16, 2, 64, dtype, gen)
    q, k, v = packed(21, 8, 2, 64, dtype, 9)
    mask = ref.random_mask(drafts, 1, gen)
    p = pool.params(8, out_dtype=dtype)
    r = ops.make_rows(21, 10)
    pool.tables[0, 2], pool.tables[0, 9], pool.tables[2, 0] = -1, pool.pages, 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def go():
        status.zero_()
        return ops.tree(p, r, q, k, v, ref.cu(drafts), mask, pool.k, pool.v, pool.tables, pool.context,
                        dev_status=status)
    out = go()
    assert int(status.item()) == ops.PA_DEV_BAD_PAGE
    want, tol = ref.tree_ref(q, k, v, drafts, mask, *pool.kv, pool.tables, lens, p.scale, dtype, dtype)
    ref.assert_close(out, want, tol)
    pool.context[1] = pool.blocks * 16 + 1
    out = go()
    assert int(status.item()) == ops.PA_DEV_BAD_PAGE | ops.PA_DEV_BAD_LEN
    assert (out[10:14] == 0).all()
    want[10:14] = 0
    ref.assert_close(out, want, tol)
    pool.context[1] = -3
    assert (go()[10:14] == 0).all()


def test_tree_replays_share_a_workspace():
    """Two captured calls of different shapes, one workspace, replayed in turn; bits repeat."""
    kw = dict(dtype="bf16", out_dtype="bf16", hq=16, hkv=4, d=128, page=32)
    made = [run_tree([900, 33], [20, 5], seed=3, **kw), run_tree([64, 2000, 7], [1, 64, 30], seed=4, **kw)]
    need = max(ops.tree_workspace_size(m[1], m[2]) for m in made)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for pool, p, r, q, k, v, c, mask, first in made:
        out = torch.zeros_like(first)
        ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for out in outs:
            out.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for m, out in zip(made, outs):
            assert torch.equal(out, m[-1])


def test_two_streams_at_once():
    """A prompt and a tree on two streams, with workspaces of their own."""
    a = run_prompt([700, 300], "bf16", "bf16", 16, 4, 128)
    b = run_tree([1500, 200], [30, 64], "bf16", "bf16", 16, 4, 128, 32)
    pool, p, r, q, k, v, c, mask, want = b
    pp = ops.prompt_params(num_seqs=2, num_q_heads=16, num_kv_heads=4, head_dim=128, dtype="bf16", out_dtype="bf16")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    cu = ref.cu([700, 300])
    outs = [(torch.zeros_like(a[3]), torch.zeros_like(want)) for _ in range(4)]
    ws = torch.empty(ops.tree_workspace_size(p, r), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for x, y in outs:
        ops.prompt(pp, ops.make_rows(1000, 700), *a[:3], cu, out=x, stream=s1)
        ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, out=y, workspace=ws, stream=s2)
        got.append((x, y))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, a[3]) and torch.equal(y, want)


@pytest.mark.parametrize("op", ("prompt", "tree"))
def test_a_wait_that_runs_out_is_reported(op):
    """debug_timeout: every wait gives up before a copy is issued; the status says so and the next call is right."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "prompt":
        q, k, v = packed(200, 8, 2, 64, "bf16", 1)
        p = ops.prompt_params(num_seqs=1, num_q_heads=8, num_kv_heads=2, head_dim=64, dtype="bf16", debug_timeout=1)
        ops.prompt(p, ops.make_rows(200, 200), q, k, v, ref.cu([200]), dev_status=status)
    else:
        pool, p, r, q, k, v, c, mask, _ = run_tree([90], [5], "bf16", "f32", 8, 2, 64, 16)
        p.debug_timeout = 1
        ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, dev_status=status)
    assert int(status.item()) & ops.PA_DEV_TIMEOUT
    run_prompt([300], "bf16", "bf16", 8, 2, 64)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("n", (33, 70))
def test_prompt_many_sequences(dtype, n):
    """More sequences than a warp has lanes, some empty, some of several units."""
    run_prompt([0 if i % 5 == 3 else (i * 53) % 190 + (400 if i == 40 else 0) for i in range(n)], dtype, dtype, 8, 2, 64, pad=2)


def test_tree_bad_length_beside_bad_values():
    """A sequence whose length is refused is zeros even where its drafts' V are not finite."""
    pool, p, r, q, k, v, c, mask, clean = run_tree([60, 40], [9, 6], "bf16", "bf16", 4, 2, 64, 16)
    v[3, 0, 1] = float("nan")
    pool.context[0] = -1
    out = ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context)
    assert (out[:9] == 0).all() and torch.equal(out[9:], clean[9:])


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_tree_workspace_holds_nothing_over(dtype):
    """A workspace full of another call's pieces gives the bits that a filled one gives."""
    kw = dict(dtype=dtype, out_dtype=dtype, hq=8, hkv=2, d=64, page=16)
    a = run_tree([900, 33, 0], [20, 40, 7], seed=3, **kw)
    b = run_tree([64, 2000, 7], [33, 64, 30], seed=4, **kw)
    ws = torch.empty(max(ops.tree_workspace_size(m[1], m[2]) for m in (a, b)), dtype=torch.uint8, device="cuda")
    for m in (a, b, a, b, b):
        pool, p, r, q, k, v, c, mask, first = m
        out = ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, workspace=ws)
        assert torch.equal(out, first)
    ws.fill_(127)
    pool, p, r, q, k, v, c, mask, first = a
    assert torch.equal(ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, workspace=ws), first)


@pytest.mark.parametrize("op", ("prompt", "tree"))
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_rows_before_the_first_sequence(op, dtype):
    """Ends that start above 0: the rows before them have no part in the call."""
    lens, first, total = [40, 9], 5, 57
    q, k, v = packed(total, 4, 2, 64, dtype, 8)
    for x in (q, k, v):
        x[:first], x[first + 49:] = float("nan"), float("nan")
    c = ref.cu(lens) + first
    out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    mine = slice(first, first + 49)
    if op == "prompt":
        p = ops.prompt_params(num_seqs=2, num_q_heads=4, num_kv_heads=2, head_dim=64, dtype=dtype, out_dtype=dtype)
        ops.prompt(p, ops.make_rows(total, 40), q, k, v, c, out=out, dev_status=status)
        want, tol = ref.prompt_ref(q[mine], k[mine], v[mine], lens, p.scale, dtype, dtype)
    else:
        gen = torch.Generator().manual_seed(9)
        pool = ref.Pool([70, 3], 16, 2, 64, dtype, gen)
        p = pool.params(4, out_dtype=dtype)
        mask = ref.random_mask([first] + lens + [3], 2, gen)
        ops.tree(p, ops.make_rows(total, 40), q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, out=out,
                 dev_status=status)
        want, tol = ref.tree_ref(q[mine], k[mine], v[mine], lens, mask[mine].contiguous(), *pool.kv, pool.tables, [70, 3],
                                 p.scale, dtype, dtype)
    assert int(status.item()) == 0
    ref.assert_close(out[mine], want, tol)
    assert (out[:first] == 7.0).all() and (out[first + 49:] == 7.0).all()


@pytest.mark.parametrize("dtype", ("f32", "f16"))
def test_tree_histories_past_their_limit(dtype):
    """A block table may hold more than 2^30 tokens; a history may not be that long."""
    hq, blocks = 4, 1 << 27  # of 16 slots: 2^31
    q, k, v = packed(3, hq, 2, 64, dtype, 4)
    pool = torch.zeros(2, 16, 2, 64, dtype=ref.DT[dtype], device="cuda")
    tables = torch.zeros(1, blocks, dtype=torch.int32, device="cuda")
    p = ops.make_params(num_seqs=1, num_q_heads=hq, num_kv_heads=2, head_dim=64, page_size=16, num_pages=2,
                        max_blocks_per_seq=blocks, max_context_len=0, dtype=dtype, out_dtype=dtype)
    r, mask = ops.make_rows(3, 3), torch.ones(3, 1, dtype=torch.int32, device="cuda")
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.tree(p, r, q, k, v, ref.cu([3]), mask, pool, pool, tables, torch.tensor([n], dtype=torch.int32, device="cuda"),
                 out=out, dev_status=status)
        assert int(status.item()) == ops.PA_DEV_BAD_LEN
        assert (out == 0).all()


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("out_dtype", ("f32", None))
def test_long_prompt_with_bad_values(dtype, out_dtype):
    """Rows find the values that are not finite among many keys without the call taking hundreds of times as long."""
    n, d, out_dtype = 20000, 64, out_dtype or dtype
    q, k, v = packed(n, 2, 1, d, dtype, 6)
    p = ops.prompt_params(num_seqs=1, num_q_heads=2, num_kv_heads=1, head_dim=d, dtype=dtype, out_dtype=out_dtype)
    r, c = ops.make_rows(n, n), ref.cu([n])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def timed():
        ops.prompt(p, r, q, k, v, c, dev_status=status)
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        out = ops.prompt(p, r, q, k, v, c, dev_status=status)
        e[1].record()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return out, e[0].elapsed_time(e[1])
    clean, t0 = timed()
    v[3, 0, 7] = float("nan")
    v[40:, 0, 9] = float("inf")       # a dim that overflows from there on
    v[9000, 0, 40] = -float("inf")
    v[9500, 0, 40] = float("inf")     # and their sum
    out, t1 = timed()
    want = clean.clone()
    want[3:, :, 7], want[40:, :, 9] = float("nan"), float("inf")
    want[9000:, :, 40] = -float("inf")
    want[9500:, :, 40] = float("nan")
    same = (out == want) | (out.isnan() & want.isnan())
    assert same.all(), f"{int((~same).sum())} elements"
    assert t1 < 60 * t0 + 5, f"{t0} ms, {t1} ms with values that are not finite"
    v[5:] = float("nan")              # all that a bad token leaves in the layers behind it
    out, t1 = timed()
    assert out[5:].isnan().all()
    assert t1 < 60 * t0 + 5, f"{t0} ms, {t1} ms with NaNs behind row 5"


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("n", (2, 40))
def test_prompt_graph_for_many_more_rows(dtype, n):
    """A graph captured for 6000 rows, replayed with few, with none, and with all of them."""
    hq, hkv, d, total = 6, 3, 64, 6000
    q, k, v = packed(total, hq, hkv, d, dtype, n)
    p = ops.prompt_params(num_seqs=n, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=dtype, out_dtype=dtype)
    r, c = ops.make_rows(total, total), ref.cu([0] * n)
    out, status = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.prompt(p, r, q, k, v, c, out=out, dev_status=status)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.prompt(p, r, q, k, v, c, out=out, dev_status=status)
    for lens in ([0] * (n - 1) + [70], [0] * n, [33] * n, [total - n + 1] + [1] * (n - 1), [1] * n):
        c.copy_(ref.cu(lens))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        m = sum(lens)
        assert (out[m:] == 7.0).all()
        if m:
            want, tol = ref.prompt_ref(q[:m], k[:m], v[:m], lens, p.scale, dtype, dtype)
            ref.assert_close(out[:m], want, tol, f"{lens[:2]}")


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("hq,hkv", [(16, 8), (32, 8)])
def test_prompt_few_and_many_units(dtype, out_dtype, d, hq, hkv):
    """Of the 16-bit kernel: units of one tile of rows, and of two."""
    run_prompt([1100, 5, 700], dtype, out_dtype, hq, hkv, d, pad=1)
