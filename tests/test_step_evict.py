"""pa_evict against its definition, key by key: what stays, in which order, and every row of the pool."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import Pool

pytestmark = pytest.mark.gpu


def stays(w, L, n, first, recent):
    r = min(recent, n)
    f = min(first, n - r)
    rank = {j: (-math.inf if math.isnan(w[j]) else w[j]) for j in range(f, L - r)}
    top = sorted(rank, key=lambda j: (-rank[j], j))[:n - r - f]
    return list(range(f)) + sorted(top) + list(range(L - r, L))


def check(pool, weights, keep, first, recent, refcounts=None, whole=(), status_is=0, lens=None):
    """Runs a call and compares all it writes; sequences in `whole` keep all, those with lens None are refused."""
    lens = pool.lens if lens is None else lens
    context = torch.tensor([99999999 if n is None else n for n in lens], dtype=torch.int32, device="cuda")
    want_kv = [x.clone() for x in pool.kv]
    slots = pool.blocks * pool.page
    out, kept = torch.full_like(weights, 7.0), torch.full(weights.shape, 7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new_lens = torch.full((len(lens),), 7, dtype=torch.int32, device="cuda")
    p = pool.params(pool.hkv)
    table = pool.tables.cpu().tolist()
    want_new = []
    want_kept, want_out = kept.clone(), out.clone()
    host = weights.cpu().tolist()
    for s, L in enumerate(lens):
        if L is None:
            want_new.append(-1)
            continue
        cut = 0 <= keep[s] < L and s not in whole
        n = keep[s] if cut else L
        want_new.append(n if cut else -1)
        for g in range(pool.hkv):
            mine = stays(host[s][g], L, n, first, recent) if cut else list(range(L))
            assert len(mine) == n
            index = torch.tensor(mine, dtype=torch.long, device="cuda")
            want_kept[s, g, :n] = index.to(torch.int32)
            want_out[s, g, :n] = weights[s, g, index]
            moves = [(j, i) for j, i in enumerate(mine) if i != j and 0 <= table[s][j // pool.page] < pool.pages and 0 <= table[s][i // pool.page] < pool.pages]
            if not moves:
                continue
            to, fr = (torch.tensor(x, device="cuda") for x in zip(*moves))
            t = pool.tables[s].long()
            for new, old in zip(want_kv, pool.kv):
                new[t[to // pool.page], to % pool.page, g] = old[t[fr // pool.page], fr % pool.page, g]
    ops.evict(p, pool.k, pool.v, pool.tables, context, weights, torch.tensor(keep, dtype=torch.int32, device="cuda"), out, kept, new_lens,
              first=first, recent=recent, refcounts=refcounts, dev_status=status)
    assert int(status) == status_is and new_lens.tolist() == want_new
    assert torch.equal(kept, want_kept)
    assert torch.equal(out.nan_to_num(5.0), want_out.nan_to_num(5.0))
    for got, want in zip(pool.kv, want_kv):
        assert torch.equal(got.nan_to_num(5.0), want.nan_to_num(5.0))
    assert slots == weights.shape[2]


CASES = [  # lens, keep, first, recent, hkv, d, page, head_major
    ((1, 2, 3, 17, 0), (0, 1, 5, 16, 3), 0, 0, 2, 64, 16, False),
    ((300, 257, 290, 64), (256, 192, 280, 64), 4, 32, 3, 64, 16, True),
    ((1000, 999, 513, 31), (999, 100, 512, -1), 1, 1, 1, 128, 32, False),
    ((5000, 4097), (1, 4096), 4, 64, 2, 128, 32, False),
    ((200, 100), (50, 60), 1000, 0, 4, 64, 32, True),
    ((200, 100), (50, 60), 0, 1000, 4, 256, 32, False),
    ((200, 100), (50, 60), 20, 30, 5, 128, 16, False),
    ((20000,), (1500,), 4, 100, 2, 64, 32, False),
    ((70000, 3), (69000, 2), 4, 100, 1, 64, 32, False),
    ((400,) * 40, tuple(range(0, 400, 10)), 2, 8, 8, 64, 16, False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_evict(case, dtype):
    lens, keep, first, recent, hkv, d, page, head_major = CASES[case]
    gen = torch.Generator().manual_seed(300 + case)
    pool = Pool(list(lens), page, hkv, d, dtype, gen, head_major=head_major, room=1)
    weights = torch.randn(len(lens), hkv, pool.blocks * page, generator=gen).exp().cuda()
    weights[:, :, ::3] = weights[:, :, ::3].round()  # equal ones
    check(pool, weights, keep, first, recent)


@pytest.mark.parametrize("kind", ["equal", "special", "tiny", "negative"])
def test_orders(kind):
    gen = torch.Generator().manual_seed(17)
    pool = Pool([700, 1500], 16, 3, 64, "f16", gen)
    w = torch.randn(2, 3, pool.blocks * 16, generator=gen)
    if kind == "equal":
        w[:] = 0.5
    elif kind == "special":
        for i, x in enumerate((math.inf, -math.inf, math.nan, 0.0, -0.0, 3.4e38, -3.4e38)):
            w[:, :, i::9] = x
    elif kind == "tiny":
        w = w * 1e-44
    else:
        w = -w.abs()
    check(pool, w.cuda(), (350, 200), 3, 5)


def test_nothing_but_what_stays_anyway():
    pool = Pool([64, 64], 16, 2, 64, "bf16", torch.Generator().manual_seed(1))
    w = torch.full((2, 2, 64), math.nan, device="cuda")
    check(pool, w, (10, 0), 4, 6)


def test_shared_pages_lengths_and_pages_outside_the_pool():
    gen = torch.Generator().manual_seed(2)
    pool = Pool([100, 100, 100, 100], 16, 2, 64, "bf16", gen)
    w = torch.rand(4, 2, pool.blocks * 16, generator=gen).cuda()
    ref = torch.zeros(pool.pages, dtype=torch.int32, device="cuda")
    ref[pool.tables[pool.tables >= 0].long()] = 1
    ref[pool.tables[0, 2].long()] = 2  # would be written
    ref[pool.tables[1, 0].long()] = 2  # inside the first keys, which stay
    ref[pool.tables[2, 6].long()] = 2  # behind what is kept
    check(pool, w, (60, 60, 60, 60), 16, 8, refcounts=ref, whole=(0,), status_is=ops.PA_DEV_SHARED_PAGE)
    pool = Pool([100, 100, 100, 100], 16, 2, 64, "bf16", gen)
    pool.tables[0, 1], pool.tables[1, 6] = -1, pool.pages
    check(pool, w, (60, 60, 60, 60), 0, 8, status_is=ops.PA_DEV_BAD_PAGE)
    pool = Pool([100, 100, 100, 100], 16, 2, 64, "bf16", gen)
    check(pool, w, (60, 60, 60, 60), 0, 8, status_is=ops.PA_DEV_BAD_LEN, lens=[100, None, 90, 100])


def test_captured_and_replayed():
    gen = torch.Generator().manual_seed(3)
    pool = Pool([500, 300], 32, 2, 128, "bf16", gen)
    p = pool.params(2)
    w, keep = torch.rand(2, 2, pool.blocks * 32, generator=gen).cuda(), torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    out, kept, new = torch.zeros_like(w), torch.zeros(w.shape, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    context = torch.zeros(2, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            ops.evict(p, pool.k, pool.v, pool.tables, context, w, keep, out, kept, new, first=2, recent=3)
    for lens, n in (([500, 300], [100, 299]), ([90, 20], [64, 20])):
        context.copy_(torch.tensor(lens, dtype=torch.int32))
        keep.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for s in range(2):
            cut = n[s] < lens[s]
            assert int(new[s]) == (n[s] if cut else -1)
            for g in range(2):
                want = stays(w[s, g].tolist(), lens[s], n[s], 2, 3) if cut else list(range(lens[s]))
                assert kept[s, g, :len(want)].tolist() == want


def test_pages_far_apart():
    """Pages whose offsets, in elements, pass 32 bits."""
    gen = torch.Generator().manual_seed(4)
    pages, page, hkv, d, stride = 36, 16, 2, 64, 1 << 26
    pools = [torch.zeros(pages * stride, dtype=torch.bfloat16, device="cuda").as_strided((pages, page, hkv, d), (stride, hkv * d, d, 1)) for _ in range(2)]
    for x in pools:
        x.copy_(torch.randn(pages, page, hkv, d, generator=gen))
    old = [x.clone() for x in pools]
    table = torch.randperm(pages, generator=gen).to(torch.int32).cuda().reshape(1, pages)
    p = ops.make_params(num_seqs=1, num_q_heads=2, num_kv_heads=hkv, head_dim=d, page_size=page, num_pages=pages, max_blocks_per_seq=pages,
                        max_context_len=pages * page, dtype="bf16", strides=(stride, 0, 0))
    w = torch.rand(1, hkv, pages * page, generator=gen).cuda()
    _, kept, new = ops.evict(p, pools[0], pools[1], table, torch.tensor([570], dtype=torch.int32, device="cuda"), w,
                             torch.tensor([300], dtype=torch.int32, device="cuda"), first=3, recent=10)
    assert new.tolist() == [300]
    to = torch.arange(300, device="cuda")
    t = table[0].long()
    for g in range(hkv):
        src = torch.tensor(stays(w[0, g].tolist(), 570, 300, 3, 10), device="cuda")
        assert torch.equal(kept[0, g, :300].long(), src)
        for x, y in zip(pools, old):
            assert torch.equal(x[t[to // page], to % page, g], y[t[src // page], src % page, g])


@pytest.mark.parametrize("blocks,L", [(2048, 30000), (20000, 300000)])
def test_tables_longer_than_a_cta_holds(blocks, L):
    """Clusters of two and eight CTAs, the latter with more weights than their registers hold."""
    page, pages = 16, -(-L // 16)
    p = ops.make_params(num_seqs=1, num_q_heads=1, num_kv_heads=1, head_dim=64, page_size=page, num_pages=pages, max_blocks_per_seq=blocks,
                        max_context_len=blocks * page, dtype="bf16")
    gen = torch.Generator().manual_seed(5)
    pool = [torch.randn(pages, page, 1, 64, generator=gen).to(torch.bfloat16).cuda() for _ in range(2)]
    old = [x.clone() for x in pool]
    table = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda")
    table[0, :pages] = torch.randperm(pages, generator=gen).to(torch.int32).cuda()
    w = (torch.rand(1, 1, blocks * page, generator=gen) * 1000).round().cuda()  # many equal ones
    n = L // 3
    _, kept, new = ops.evict(p, pool[0], pool[1], table, torch.tensor([L], dtype=torch.int32, device="cuda"), w,
                             torch.tensor([n], dtype=torch.int32, device="cuda"), first=5, recent=77)
    src = torch.tensor(stays(w[0, 0].tolist(), L, n, 5, 77), device="cuda")
    assert new.tolist() == [n] and torch.equal(kept[0, 0, :n].long(), src)
    to, t = torch.arange(n, device="cuda"), table[0].long()
    for x, y in zip(pool, old):
        assert torch.equal(x[t[to // page], to % page], y[t[src // page], src % page])
