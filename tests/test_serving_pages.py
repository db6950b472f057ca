"""The K/V store and the page operations on the GPU against host models, and
a serving step put together from all of them."""
from __future__ import annotations

import random

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def params(seqs, pages, blocks, page=16, hkv=2, d=64, dtype="bf16", **kw):
    return ops.make_params(num_seqs=seqs, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, page_size=page,
                           num_pages=pages, max_blocks_per_seq=blocks, max_context_len=blocks * page, dtype=dtype, **kw)


# ---- store ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ("f32", "f16", "bf16"))
@pytest.mark.parametrize("page,hkv,d,head_major", [(16, 1, 64, False), (32, 8, 128, False), (16, 3, 256, True)])
@pytest.mark.parametrize("pick", (False, True))
def test_store(dtype, page, hkv, d, head_major, pick):
    gen = torch.Generator().manual_seed(2)
    lens, rows = [40, 7, 1, 0, 200, 33, 64], [40, 3, 1, 0, 90, 2, 0]
    pool = ref.Pool(lens, page, hkv, d, dtype, gen, head_major=head_major)
    total, pad = sum(rows), 4
    src = total + pad + (30 if pick else 0)
    wide = torch.randn((src, 2 * hkv, d), generator=gen).to(ref.DT[dtype]).cuda()
    k, v = wide[:, :hkv], wide[:, hkv:]
    index = torch.randint(0, src, (total + pad,), generator=gen).to(torch.int32).cuda() if pick else None
    want = [x.clone() for x in pool.kv]
    at = 0
    for s, n in enumerate(rows):
        for i in range(n):
            pos = lens[s] - n + i
            frm = int(index[at + i]) if pick else at + i
            for w, x in zip(want, (k, v)):
                w[pool.tables[s, pos // page], pos % page] = x[frm]
        at += n
    r = ops.make_rows(total + pad, max(rows), source_rows=src, k_stride=2 * hkv * d, v_stride=2 * hkv * d)
    status = status_word()
    ops.store(pool.params(hkv), r, k, v, ref.cu(rows), pool.k, pool.v, pool.tables, pool.context, row_index=index,
              dev_status=status)
    assert int(status.item()) == 0
    for got, w in zip(pool.kv, want):
        assert torch.equal(got.nan_to_num(9.0), w.nan_to_num(9.0)) and torch.equal(got.isnan(), w.isnan())


@pytest.mark.parametrize("n", (1, 31, 32, 33, 64, 65, 1100))
def test_store_finds_the_sequence_among_many(n):
    """One row each, some none: every search depth."""
    rows = [(i * 7) % 3 for i in range(n)]
    rows[-1] = 1
    lens = [x + i % 5 for i, x in enumerate(rows)]
    gen = torch.Generator().manual_seed(n)
    pool = ref.Pool(lens, 16, 1, 64, "f32", gen)
    total = sum(rows)
    k, v = (torch.randn((total, 1, 64), generator=gen).cuda() for _ in range(2))
    ops.store(pool.params(1), ops.make_rows(total, max(rows)), k, v, ref.cu(rows), pool.k, pool.v, pool.tables,
              pool.context)
    seq = torch.repeat_interleave(torch.arange(n), torch.tensor(rows)).cuda()
    place = torch.arange(total, device="cuda") - ref.cu(rows)[seq]
    pos = pool.context[seq] - torch.tensor(rows, device="cuda")[seq] + place
    got = pool.k[pool.tables[seq, (pos // 16).long()].long(), (pos % 16).long()]
    assert torch.equal(got, k)


def test_store_refused_rows():
    gen = torch.Generator().manual_seed(5)
    pool = ref.Pool([40, 20, 20, 20], 16, 2, 64, "bf16", gen)
    k, v = (torch.randn((12, 2, 64), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    before = [x.clone() for x in (pool.k, pool.v)]
    pool.tables[1, 1] = pool.pages
    pool.context[2] = 2                                  # fewer than its rows
    pool.context[3] = pool.blocks * 16 + 1
    index = i32([0, -1, 12, 1, 2, 3, 4, 5, 6, 7, 8, 9])
    status = status_word()
    ops.store(pool.params(2), ops.make_rows(12, 3), k, v, ref.cu([3, 3, 3, 3]), pool.k, pool.v, pool.tables,
              pool.context, row_index=index, dev_status=status)
    assert int(status.item()) == ops.PA_DEV_BAD_PAGE | ops.PA_DEV_BAD_LEN | ops.PA_DEV_BAD_INDEX
    before[0][pool.tables[0, 2].long(), 5], before[1][pool.tables[0, 2].long(), 5] = k[0], v[0]  # position 37
    for got, w in zip((pool.k, pool.v), before):
        assert torch.equal(got.nan_to_num(9.0), w.nan_to_num(9.0))


def test_store_leaves_rows_before_the_first_sequence():
    gen = torch.Generator().manual_seed(15)
    pool = ref.Pool([20, 5], 16, 2, 64, "bf16", gen)
    k, v = (torch.randn((9, 2, 64), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    want = [x.clone() for x in pool.kv]
    for s, (row, n, L) in enumerate([(3, 4, 20), (7, 1, 5)]):
        for i in range(n):
            pos = L - n + i
            for w, x in zip(want, (k, v)):
                w[pool.tables[s, pos // 16].long(), pos % 16] = x[row + i]
    status = status_word()
    ops.store(pool.params(2), ops.make_rows(9, 4), k, v, i32([3, 7, 8]), pool.k, pool.v, pool.tables, pool.context,
              dev_status=status)
    assert int(status.item()) == 0
    for got, w in zip(pool.kv, want):
        assert torch.equal(got.nan_to_num(9.0), w.nan_to_num(9.0))


# ---- bookkeeping -----------------------------------------------------------------

class Device:
    def __init__(self, seqs, pages, blocks, page):
        self.p = params(seqs, pages, blocks, page)
        self.ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.tables = torch.full((seqs, blocks), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.pairs = torch.full((seqs, 2), 5, dtype=torch.int32, device="cuda")
        self.ws = torch.full((ops.pages_workspace_size(self.p),), 255, dtype=torch.uint8, device="cuda")
        self.status = status_word()
        self.model = ref.PageModel(self.ref.tolist(), self.tables.tolist(), self.lens.tolist(), page)

    def take(self):
        s = int(self.status.item())
        self.status.zero_()
        return s

    def resize(self, new):
        ops.pages_resize(self.p, self.ref, self.tables, self.lens, i32(new), self.pairs, self.ws, dev_status=self.status)
        pairs, short = self.model.resize(new)
        assert self.pairs.tolist() == pairs
        assert self.take() == (ops.PA_DEV_NO_PAGES if short else 0)
        self.check()
        return short

    def fork(self, src, dst):
        ops.pages_fork(self.p, self.ref, self.tables, self.lens, i32(src), i32(dst), dev_status=self.status)
        self.model.fork(src, dst)
        assert self.take() == 0
        self.check()

    def compact(self, most):
        pairs = torch.full((most, 2), 5, dtype=torch.int32, device="cuda")
        n = torch.full((1,), 99, dtype=torch.int32, device="cuda")
        ops.pages_compact(self.p, self.ref, self.tables, self.lens, pairs, n, self.ws, dev_status=self.status)
        want, moved = self.model.compact(most)
        assert pairs.tolist() == want and int(n.item()) == moved and self.take() == 0
        self.check()

    def check(self):
        assert self.lens.tolist() == self.model.lens
        assert self.ref.tolist() == self.model.ref
        page = self.model.page
        for s, (a, b) in enumerate(zip(self.tables.tolist(), self.model.tables)):
            n = -(-self.model.lens[s] // page)
            assert a[:n] == b[:n], f"table of sequence {s}"


@pytest.mark.parametrize("seqs,pages,blocks,page", [(1, 1, 1, 16), (5, 40, 12, 16), (40, 300, 20, 32),
                                                    (300, 5000, 40, 16), (700, 9000, 30, 32)])
def test_pages_random_walk(seqs, pages, blocks, page):
    rng = random.Random(seqs)
    d = Device(seqs, pages, blocks, page)
    top = blocks * page
    for step in range(12):
        lens = d.model.lens
        kind = rng.random()
        if kind < 0.6 or step == 0:
            new = [rng.choice([-1, -1, 0, rng.randint(0, top), min(top, n + rng.randint(0, 2 * page)), n]) for n in lens]
            d.resize(new)
        elif kind < 0.8:
            empty = [s for s, n in enumerate(lens) if n == 0]
            some = [s for s, n in enumerate(lens) if n]
            rng.shuffle(empty)
            dst = empty[:len(empty) // 2 + 1]
            if dst and some:
                d.fork([rng.choice(some) for _ in dst], dst)
        else:
            d.compact(rng.choice([0, 1, 7, pages]))
    d.compact(pages)
    live = sum(1 for r in d.model.ref if r)
    assert d.ref.tolist() == d.model.ref and all(d.model.ref[:live])
    d.resize([0] * seqs)
    assert int(d.ref.abs().sum()) == 0


def test_resize_when_pages_run_out():
    """In order: the first that does not fit and all that ask after it stay as they were; shrinking goes on."""
    d = Device(4, 10, 10, 16)
    d.resize([64, 33, 0, 0])
    assert d.resize([-1, 16, 80, 16])  # five asked for of three free; one released, but not yet free
    assert d.model.lens == [64, 16, 0, 0]
    assert not d.resize([-1, -1, 64, 16])


def test_growing_a_shared_page_copies_it():
    d = Device(3, 12, 4, 16)
    d.resize([20, 0, 0])
    d.fork([0, 0], [1, 2])
    d.resize([21, 21, -1])
    assert [p for p in d.model.tables[0][:2]] != d.model.tables[1][:2]
    d.resize([21, 21, 10])  # shrunk into a shared page: it gets its own
    d.resize([0, 0, 0])


def test_fork_and_resize_refusals():
    d = Device(6, 40, 4, 16)
    d.resize([20, 30, 0, 0, 0, 0])
    before = [x.tolist() for x in (d.ref, d.tables, d.lens)]
    for src, dst, bit in (([0], [1], 32), ([0], [6], 32), ([-1], [2], 32), ([6], [2], 32), ([2], [2], 32),
                          ([2, 0], [3, 2], 32)):
        if dst == [3, 2]:  # the second pair is good: its source is no destination
            ops.pages_fork(d.p, d.ref, d.tables, d.lens, i32(src), i32(dst), dev_status=d.status)
            assert d.take() == bit and d.lens.tolist() == [20, 30, 20, 0, 0, 0]
            ops.pages_resize(d.p, d.ref, d.tables, d.lens, i32([-1, -1, 0, -1, -1, -1]), d.pairs, d.ws)
        else:
            ops.pages_fork(d.p, d.ref, d.tables, d.lens, i32(src), i32(dst), dev_status=d.status)
            assert d.take() == bit
        assert d.ref.tolist() == before[0] and d.lens.tolist() == before[2]
    ops.pages_fork(d.p, d.ref, d.tables, d.lens, i32([0, 1]), i32([2, 2]), dev_status=d.status)  # the first wins
    assert d.take() == 32 and d.lens.tolist() == [20, 30, 20, 0, 0, 0]
    ops.pages_resize(d.p, d.ref, d.tables, d.lens, i32([-1, 65, 1 << 30, -1, -1, -1]), d.pairs, d.ws,
                     dev_status=d.status)
    assert d.take() == ops.PA_DEV_BAD_LEN and d.lens.tolist() == [20, 30, 20, 0, 0, 0]
    assert d.pairs.tolist() == [[-1, -1]] * 6
    d.tables[1, 1] = 40  # outside the pool: passed over when it is released
    held = int(d.ref.sum())
    ops.pages_resize(d.p, d.ref, d.tables, d.lens, i32([-1, 0, -1, -1, -1, -1]), d.pairs, d.ws, dev_status=d.status)
    assert d.take() == ops.PA_DEV_BAD_PAGE and int(d.ref.sum()) == held - 1
    d.lens[0] = -4
    n = i32([0])
    ops.pages_compact(d.p, d.ref, d.tables, d.lens, d.pairs, n, d.ws, dev_status=d.status)
    assert d.take() == ops.PA_DEV_BAD_LEN


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("page,hkv,d,head_major", [(16, 1, 64, False), (32, 8, 128, False), (32, 5, 256, True)])
def test_copy(dtype, page, hkv, d, head_major):
    gen = torch.Generator().manual_seed(1)
    pages = 30
    pool = ref.Pool([page * pages], page, hkv, d, dtype, gen, spare=0, head_major=head_major)
    p = pool.params(hkv)
    pairs = [[3, 7], [-1, 4], [3, 8], [5, -1], [-1, -1], [2, 2], [0, 29], [3, 30], [30, 11], [9, 1]]
    want = [x.clone() for x in pool.kv]
    for w, x in zip(want, pool.kv):
        for a, b in ((3, 7), (3, 8), (0, 29), (9, 1)):
            w[b] = x[a]
    status = status_word()
    ops.pages_copy(p, pool.k, pool.v, i32(pairs), dev_status=status)
    assert int(status.item()) == ops.PA_DEV_BAD_INDEX
    for got, w in zip(pool.kv, want):
        assert torch.equal(got, w)


def test_copy_flags_a_pair_outside_the_pool_that_goes_nowhere():
    pool = torch.ones(3, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    p = params(1, 3, 1)
    for pair, want in (([7, 7], ops.PA_DEV_BAD_INDEX), ([1, 1], 0), ([-1, 9], 0), ([0, 3], ops.PA_DEV_BAD_INDEX)):
        status = status_word()
        ops.pages_copy(p, pool, pool.clone(), i32([pair]), dev_status=status)
        assert int(status.item()) == want, pair
        assert (pool == 1).all()


def test_page_calls_replay():
    """A step captured once (grow, copy, compact, copy) and replayed follows the lengths that it finds."""
    d = Device(8, 64, 6, 16)
    d.resize([30, 16, 50, 0, 70, 1, 0, 33])
    d.fork([0, 2], [3, 6])
    k, v = (torch.randn(64, 16, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    grow, moves, n = i32([31, 17, 51, 40, 71, 2, 51, 34]), torch.zeros(64, 2, dtype=torch.int32, device="cuda"), i32([0])

    def step():
        ops.pages_resize(d.p, d.ref, d.tables, d.lens, grow, d.pairs, d.ws)
        ops.pages_copy(d.p, k, v, d.pairs)
        ops.pages_compact(d.p, d.ref, d.tables, d.lens, moves, n, d.ws)
        ops.pages_copy(d.p, k, v, moves)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for new in ([31, 17, 51, 40, 71, 2, 51, 34], [0, 18, 52, -1, 0, 3, 52, 35], [90, 0, 53, 96, 96, 96, 0, 36]):
        grow.copy_(i32(new))
        g.replay()
        torch.cuda.synchronize()
        d.model.resize(new)
        d.model.compact(64)
        d.check()


# ---- a serving step ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_a_serving_step(dtype):
    """Reserve, prompt, store, fork, grow with copy-on-write, draft a chain,
    accept part of it by index, compact, decode: what decode then reads is the
    sequence that a prompt call sees whole."""
    gen = torch.Generator().manual_seed(8)
    hq, hkv, d, page, pages, blocks = 8, 2, 64, 16, 80, 10
    lens = [37, 64, 5]
    n = 5  # three requests, two forks
    p = ops.make_params(num_seqs=n, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page, num_pages=pages,
                        max_blocks_per_seq=blocks, max_context_len=blocks * page, dtype=dtype)

    def normal(*shape):
        return torch.randn(shape, generator=gen).to(ref.DT[dtype]).cuda()
    counts = torch.zeros(pages, dtype=torch.int32, device="cuda")
    counts[:20] = 1  # somebody else's pages
    tables = torch.full((n, blocks), -1, dtype=torch.int32, device="cuda")
    context = torch.zeros(n, dtype=torch.int32, device="cuda")
    pairs = torch.zeros(n, 2, dtype=torch.int32, device="cuda")
    k_cache, v_cache = (torch.full((pages, page, hkv, d), float("nan"), dtype=ref.DT[dtype], device="cuda")
                        for _ in range(2))
    status = status_word()

    ops.pages_resize(p, counts, tables, context, i32(lens + [0, 0]), pairs, dev_status=status)
    q, k, v = normal(sum(lens), hq, d), normal(sum(lens), hkv, d), normal(sum(lens), hkv, d)
    rows = ops.make_rows(sum(lens), max(lens))
    c = ref.cu(lens + [0, 0])
    out = ops.prompt(p, rows, q, k, v, c, dev_status=status)
    want, tol = ref.prompt_ref(q, k, v, lens, p.scale, dtype, "f32")
    ref.assert_close(out, want, tol, "prompt")
    ops.store(p, rows, k, v, c, k_cache, v_cache, tables, context, dev_status=status)
    ops.pages_fork(p, counts, tables, context, i32([0, 1]), i32([3, 4]), dev_status=status)
    whole = [(k[a:b], v[a:b]) for a, b in ((0, 37), (37, 101), (101, 106), (0, 37), (37, 101))]

    # every sequence drafts four in a chain and takes its first, third and fourth as a new tail
    drafts = [4] * n
    dq, dk, dv = normal(4 * n, hq, d), normal(4 * n, hkv, d), normal(4 * n, hkv, d)
    chain = torch.tensor([[1], [3], [7], [15]] * n, dtype=torch.int32, device="cuda")
    out = ops.tree(p, ops.make_rows(4 * n, 4), dq, dk, dv, ref.cu(drafts), chain, k_cache, v_cache, tables, context,
                   dev_status=status)
    want, tol = ref.tree_ref(dq, dk, dv, drafts, chain, k_cache, v_cache, tables, context.tolist(), p.scale, dtype, "f32")
    ref.assert_close(out, want, tol, "tree")
    grown = [len(a) + 3 for a, _ in whole]
    ops.pages_resize(p, counts, tables, context, i32(grown), pairs, dev_status=status)
    ops.pages_copy(p, k_cache, v_cache, pairs, dev_status=status)
    accepted = [4 * s + i for s in range(n) for i in (0, 2, 3)]
    ops.store(p, ops.make_rows(3 * n, 3, source_rows=4 * n), dk, dv, ref.cu([3] * n), k_cache, v_cache, tables, context,
              row_index=i32(accepted), dev_status=status)
    whole = [(torch.cat([a, dk[[4 * s, 4 * s + 2, 4 * s + 3]]]), torch.cat([b, dv[[4 * s, 4 * s + 2, 4 * s + 3]]]))
             for s, (a, b) in enumerate(whole)]
    ops.pages_resize(p, counts, tables, context, i32([-1, 0, -1, -1, -1]), pairs, dev_status=status)  # request 1 ends
    counts[:20] = 0
    moves, moved = torch.zeros(pages, 2, dtype=torch.int32, device="cuda"), i32([0])
    ops.pages_compact(p, counts, tables, context, moves, moved, dev_status=status)
    ops.pages_copy(p, k_cache, v_cache, moves, dev_status=status)
    assert int(moved.item()) > 0
    live = int((counts > 0).sum())
    assert (counts[:live] > 0).all()

    keep = [0, 2, 3, 4]
    tail = normal(len(keep), hq, d)
    pd = ops.make_params(num_seqs=len(keep), num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page,
                         num_pages=pages, max_blocks_per_seq=blocks, max_context_len=blocks * page, dtype=dtype)
    got = ops.decode(pd, tail, k_cache, v_cache, tables[keep].contiguous(), context[keep].contiguous(), dev_status=status)
    assert int(status.item()) == 0
    for i, s in enumerate(keep):
        a, b = whole[s]
        see = torch.ones(1, len(a), dtype=torch.bool, device="cuda")
        for h in range(hq):
            g = h // (hq // hkv)
            w, wt = ref.attend(tail[i:i + 1, h].double(), a[:, g].double(), b[:, g].double(), see, p.scale)
            t = ref.bound(w, wt, tail[i:i + 1, h].double(), a[:, g].double(), p.scale, len(a), dtype, "f32")
            ref.assert_close(got[i:i + 1, h], w, t, f"decode {s} {h}")
