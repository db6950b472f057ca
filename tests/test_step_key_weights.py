"""pa_key_weights against softmax sums in 64 bits."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import DT, Pool, assert_close, cu

pytestmark = pytest.mark.gpu


def reference(q, rows, pool, weights, decay, scale):
    """(weights, bound).  A score is an fp32 dot product of D terms, off by
    D 2^-23 sum|q||k| at most (2^-23: the tensor cores may truncate), and so is
    its weight, relatively, with 2^-17 for the exponentials; numerator and
    denominator both, hence twice.  Adding n terms in fp32 adds n 2^-23, of the
    keys in the denominator and of the columns in the sum."""
    want, tol = weights.double().clone(), torch.full(weights.shape, 1e-30, dtype=torch.float64, device="cuda")
    k, group, at = pool.kv[0], q.shape[1] // pool.hkv, 0
    for s, (n, L) in enumerate(zip(rows, pool.lens)):
        spot = torch.arange(L, device="cuda")
        entry = pool.tables[s].long()[spot // pool.page] if L else spot
        there = (entry >= 0) & (entry < pool.pages)
        see = (spot[None] <= torch.arange(L - n, L, device="cuda")[:, None]) & there[None]
        for g in range(pool.hkv if n else 0):
            kk = k[entry.clamp(0, pool.pages - 1), spot % pool.page, g].double()
            kk[~there] = 0
            got = torch.zeros(L, dtype=torch.float64, device="cuda")
            size = 0.0
            for h in range(g * group, (g + 1) * group):
                qq = q[at:at + n, h].double()
                x = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
                got += torch.softmax(x, 1).nan_to_num(0.0).sum(0)
                size = max(size, float((qq.abs() @ kk.abs().T).nan_to_num(0.0).max()) * scale)
            rel = 2 * (q.shape[-1] * 2.0 ** -23 * size + 2.0 ** -17) + (L + n * group + 4) * 2.0 ** -23
            old = want[s, g, :L].clone()
            old[L - n:] = 0
            old = decay * old if decay else torch.zeros_like(old)
            want[s, g, :L] = got + old
            tol[s, g, :L] = rel * got + 2.0 ** -22 * (old.abs() + got) + 1e-30
        at += n
    return want, tol


def fresh(pool, gen):
    return torch.rand(len(pool.lens), pool.hkv, pool.blocks * pool.page, generator=gen).cuda()


CASES = [  # rows, history, hq, hkv, d, page, decay, head_major
    ((1, 1, 1, 1), (0, 31, 32, 700), 12, 3, 64, 16, 1.0, False),
    ((1, 0, 1), (3253, 5, 129), 40, 8, 128, 32, 0.5, False),
    ((1,) * 9, (0, 1, 15, 16, 17, 127, 128, 129, 1000), 16, 1, 128, 16, 1.0, True),
    ((2, 1, 5), (64, 300, 0), 4, 4, 64, 32, 0.0, False),
    ((3, 1), (900, 2000), 10, 2, 128, 32, 1.0, False),
    ((7, 26, 64, 1, 0, 13), (100, 1000, 33, 4095, 50, 0), 8, 2, 128, 32, 0.9375, False),
    ((33, 1, 100), (0, 0, 37), 5, 5, 64, 16, 1.0, True),
    ((300, 1, 129), (0, 500, 1), 16, 2, 128, 32, 1.0, False),
    ((511,), (1,), 3, 1, 128, 16, 0.0, False),
    ((700, 65), (60, 900), 8, 8, 64, 32, 1.0, False),
    ((8, 9, 1), (3000, 2, 555), 16, 4, 128, 32, 1.0, False),
    ((66, 33), (0, 1500), 2, 2, 64, 16, 0.5, False),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_key_weights(case, dtype):
    rows, history, hq, hkv, d, page, decay, head_major = CASES[case]
    gen = torch.Generator().manual_seed(200 + case)
    before, pad = (2, 3) if case % 2 else (0, 0)
    total, wide = before + sum(rows) + pad, hq * d + 32
    lens = [h + n for h, n in zip(history, rows)]
    pool = Pool(lens, page, hkv, d, dtype, gen, head_major=head_major, room=1)
    q = (2 * torch.randn(total, wide, generator=gen)).to(DT[dtype]).cuda()[:, :hq * d].unflatten(1, (hq, d))
    weights = fresh(pool, gen)
    for s, n in enumerate(rows):
        if n:
            weights[s, :, lens[s] - n:lens[s]] = float("nan")  # not read
    if decay == 0:
        weights[:] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p, r = pool.params(hq, out_dtype="f32"), ops.make_rows(total, max(rows), q_stride=wide)
    clean = weights.nan_to_num(0.25)
    want, tol = reference(q[before:], rows, pool, clean, decay, p.scale)
    got = ops.key_weights(p, r, q, cu(rows) + before, pool.k, pool.tables, pool.context, weights, decay=decay, dev_status=status)
    assert int(status) == 0
    for s, (n, L) in enumerate(zip(rows, lens)):
        if n:
            assert_close(got[s, :, :L], want[s, :, :L], tol[s, :, :L], f"sequence {s}")
        assert torch.equal(got[s, :, L if n else 0:].nan_to_num(0.25), clean[s, :, L if n else 0:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 40])
def test_pages_outside_the_pool_and_bad_lengths(rows, dtype):
    gen = torch.Generator().manual_seed(7)
    lens, hq, hkv, d = [200, 90, 300, 64], 8, 2, 128
    pool = Pool(lens, 16, hkv, d, dtype, gen)
    counts = [rows] * 4
    q = torch.randn(sum(counts), hq, d, generator=gen).to(DT[dtype]).cuda()
    pool.tables[0, 3], pool.tables[0, 12] = pool.pages, -7
    if rows == 1:
        pool.tables[3, :] = -1  # a row that sees nothing
    weights = fresh(pool, gen)
    context = torch.tensor([200, rows - 1, pool.blocks * 16 + 1, 64], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    clean = weights.clone()
    p, r = pool.params(hq), ops.make_rows(sum(counts), rows)
    got = ops.key_weights(p, r, q, cu(counts), pool.k, pool.tables, context, weights, dev_status=status)
    assert int(status) == ops.PA_DEV_BAD_PAGE | ops.PA_DEV_BAD_LEN
    assert torch.equal(got[1:3], clean[1:3])
    for s in (0, 3):
        one = Pool([lens[s]], 16, hkv, d, dtype, torch.Generator().manual_seed(1))
        one.tables, one.pages, one.kv, one.lens = pool.tables[s:s + 1], pool.pages, pool.kv, [lens[s]]
        want, tol = reference(q[s * rows:(s + 1) * rows], [rows], one, clean[s:s + 1], 1.0, 1 / math.sqrt(d))
        assert_close(got[s, :, :lens[s]], want[0, :, :lens[s]], tol[0, :, :lens[s]], f"sequence {s}")


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("rows", [1, 50])
def test_values_that_are_not_finite(rows, dtype):
    """A NaN or +infinity reaches the weights of the rows that see it; -infinity weighs nothing."""
    gen = torch.Generator().manual_seed(8)
    L, hq, hkv, d = 300, 4, 2, 64
    pool = Pool([L, L, L], 16, hkv, d, dtype, gen)
    q = torch.randn(3 * rows, hq, d, generator=gen).to(DT[dtype]).cuda()
    q[..., 0] = q[..., 0].abs() + 0.5
    bad = L - 20
    for s, value in enumerate((math.nan, math.inf, -math.inf)):
        page, slot = int(pool.tables[s, bad // 16]), bad % 16
        pool.kv[0][page, slot, 0, :] = 0
        pool.kv[0][page, slot, 0, 0] = value
    weights = torch.zeros(3, hkv, pool.blocks * 16, device="cuda")
    p, r = pool.params(hq), ops.make_rows(3 * rows, rows)
    got = ops.key_weights(p, r, q, cu([rows] * 3), pool.k, pool.tables, pool.context, weights, decay=0.0)
    want, tol = reference(q, [rows] * 3, pool, weights, 0.0, 1 / math.sqrt(d))
    assert_close(got[:, 1, :L], want[:, 1, :L], tol[:, 1, :L], "the other head")
    assert got[:2, 0, :bad + 1].isnan().all()
    if rows > 20:  # keys behind the bad one gather from rows that see it alone
        assert got[:2, 0, bad:L].isnan().all()
    assert_close(got[2, 0, :L], want[2, 0, :L], tol[2, 0, :L], "-infinity")
    assert float(got[2, 0, bad]) == 0.0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_workspace_replayed_with_other_lengths(dtype):
    """A captured call takes what the lengths, rows and tables say at each replay, and its workspace holds nothing."""
    gen = torch.Generator().manual_seed(9)
    hq, hkv, d, page = 8, 2, 128, 16
    pool = Pool([500, 400, 77], page, hkv, d, dtype, gen)
    p, r = pool.params(hq), ops.make_rows(64, 40)
    q = torch.randn(64, hq, d, generator=gen).to(DT[dtype]).cuda()
    rows, context = cu([1, 1, 1]), pool.context.clone()
    weights = torch.zeros(3, hkv, pool.blocks * page, device="cuda")
    ws = torch.full((ops.key_weights_workspace_size(p, r),), 255, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ops.key_weights(p, r, q, rows, pool.k, pool.tables, context, weights, decay=0.0, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            ops.key_weights(p, r, q, rows, pool.k, pool.tables, context, weights, decay=0.0, workspace=ws)
    torch.cuda.synchronize()
    for counts, lens in (([1, 1, 1], [500, 400, 77]), ([40, 0, 20], [333, 100, 20]), ([1, 5, 1], [1, 400, 70])):
        rows.copy_(cu(counts))
        context.copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(255)
        weights.zero_()
        graph.replay()
        torch.cuda.synchronize()
        pool.lens = lens
        want, tol = reference(q, counts, pool, torch.zeros_like(weights), 0.0, p.scale)
        assert_close(weights, want, tol + 1e-30, str(counts))


def test_two_streams_and_repeats_are_bit_equal():
    gen = torch.Generator().manual_seed(10)
    pool = Pool([3000, 1], 32, 4, 128, "bf16", gen)
    p = pool.params(16)
    for counts in ([1, 1], [200, 1]):
        r = ops.make_rows(sum(counts), max(counts))
        q = torch.randn(sum(counts), 16, 128, generator=gen).to(torch.bfloat16).cuda()
        torch.cuda.synchronize()
        outs = []
        for i in range(4):
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                w = torch.zeros(2, 4, pool.blocks * 32, device="cuda")
            outs.append(_on(st, p, r, q, cu(counts), pool, w))
        torch.cuda.synchronize()
        assert all(torch.equal(outs[0], o) for o in outs[1:])


def _on(st, p, r, q, starts, pool, w):
    st.wait_stream(torch.cuda.current_stream())
    return ops.key_weights(p, r, q, starts, pool.k, pool.tables, pool.context, w, stream=st)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 40])
def test_many_sequences(rows, dtype):
    """More sequences than a warp has lanes, some without rows, one longer than the host's bound."""
    gen = torch.Generator().manual_seed(11)
    counts = [0 if i % 7 == 3 else 1 + (i * 5) % rows for i in range(75)]
    lens = [n + (i * 37) % 400 for i, n in enumerate(counts)]
    pool = Pool(lens, 16, 2, 64, dtype, gen)
    q = torch.randn(sum(counts), 6, 64, generator=gen).to(DT[dtype]).cuda()
    weights = fresh(pool, gen)
    clean = weights.clone()
    p, r = pool.params(6), ops.make_rows(sum(counts), rows)
    want, tol = reference(q, counts, pool, clean, 0.5, p.scale)
    got = ops.key_weights(p, r, q, cu(counts), pool.k, pool.tables, pool.context, weights.clone(), decay=0.5)
    for s, (n, L) in enumerate(zip(counts, lens)):
        assert_close(got[s, :, :L], (want if n else clean.double())[s, :, :L], tol[s, :, :L], f"sequence {s}") if L else None
    p.max_context_len = 250
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bounded = ops.key_weights(p, r, q, cu(counts), pool.k, pool.tables, pool.context, weights.clone(), decay=0.5, dev_status=status)
    assert int(status) == ops.PA_DEV_BAD_LEN
    for s, L in enumerate(lens):
        assert_close(bounded[s, :, :L], (clean.double() if L > 250 else want)[s, :, :L], tol[s, :, :L], f"bounded {s}") if L else None


@pytest.mark.parametrize("rows", [1, 100])
def test_pages_far_apart(rows):
    """Pages whose offsets, in elements, pass 32 bits."""
    gen = torch.Generator().manual_seed(12)
    pages, page, hkv, d, stride = 36, 32, 2, 128, 1 << 26
    store = torch.zeros(pages * stride, dtype=torch.bfloat16, device="cuda")
    L = 300
    table = (pages - 1 - torch.arange(10, dtype=torch.int32)).cuda().reshape(1, 10)
    k = torch.randn(L, hkv, d, generator=gen).to(torch.bfloat16).cuda()
    view = store.as_strided((pages, page, hkv, d), (stride, hkv * d, d, 1))
    spot = torch.arange(L, device="cuda")
    view[table[0].long()[spot // page], spot % page] = k
    p = ops.make_params(num_seqs=1, num_q_heads=8, num_kv_heads=hkv, head_dim=d, page_size=page, num_pages=pages, max_blocks_per_seq=10,
                        max_context_len=320, dtype="bf16", strides=(stride, 0, 0))
    q = torch.randn(rows, 8, d, generator=gen).to(torch.bfloat16).cuda()
    w = torch.zeros(1, hkv, 320, device="cuda")
    ops.key_weights(p, ops.make_rows(rows, rows), q, cu([rows]), store, table, torch.tensor([L], dtype=torch.int32, device="cuda"), w, decay=0.0)
    pool = Pool([L], page, hkv, d, "bf16", gen)
    pool.tables, pool.pages, pool.kv, pool.lens = table, pages, [view], [L]
    want, tol = reference(q, [rows], pool, w * 0, 0.0, p.scale)
    assert_close(w[0, :, :L], want[0, :, :L], tol[0, :, :L])


def test_a_wait_that_runs_out_leaves_the_context_usable():
    gen = torch.Generator().manual_seed(13)
    pool = Pool([500], 16, 2, 128, "f16", gen)
    q = torch.randn(200, 8, 128, generator=gen).to(torch.float16).cuda()
    w = torch.zeros(1, 2, pool.blocks * 16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p, r = pool.params(8, debug_timeout=1), ops.make_rows(200, 200)
    ops.key_weights(p, r, q, cu([200]), pool.k, pool.tables, pool.context, w, decay=0.0, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == ops.PA_DEV_TIMEOUT
    p, w = pool.params(8), torch.zeros_like(w)
    ops.key_weights(p, r, q, cu([200]), pool.k, pool.tables, pool.context, w, decay=0.0)
    want, tol = reference(q, [200], pool, torch.zeros_like(w), 0.0, p.scale)
    assert_close(w[0, :, :500], want[0, :, :500], tol[0, :, :500])
