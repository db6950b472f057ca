"""pa_rotate: norms, rotation and store against their formulas in 64 bits."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import DT, Pool, assert_close, cu

pytestmark = pytest.mark.gpu
EPS = 1e-5


def table_of(n, rot):
    angle = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda().contiguous()


def turned(x, weight, rot, mixed, table, pos):
    """(value, bound) of rows x [n][h][d] at positions pos [n][rot / 2].

    In fp32 a norm is off by (D + 4) 2^-24 relatively at most (a sum of D
    squares, the root, the division, two products), a turned dim by three more
    roundings of each of its two terms; the result is rounded once."""
    dt, d = x.dtype, x.shape[-1]
    y = x.double()
    rel = 4 * 2.0 ** -24
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.double()
        rel += (d + 4) * 2.0 ** -24
    out, size = y.clone(), y.abs()
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if mixed else (i, half + i)
        c, s = (table.double()[pos[:, i], j][:, None] for j in (i, half + i))
        out[..., a] = c * y[..., a] - s * y[..., b]
        out[..., b] = s * y[..., a] + c * y[..., b]
        size[..., a] = (c * y[..., a]).abs() + (s * y[..., b]).abs()
        size[..., b] = (s * y[..., a]).abs() + (c * y[..., b]).abs()
    info = torch.finfo(dt)
    return out, size * rel + info.eps / 2 * (out.abs() + size * rel) + info.tiny * info.eps


CASES = [  # rows, history, hq, hkv, d, rot, mixed, sections, norms, store, k_out
    ((1, 1, 1), (0, 31, 7), 12, 3, 64, 64, False, None, "qk", True, False),
    ((5, 0, 33, 1), (0, 4, 15, 16), 4, 1, 64, 32, True, None, "", True, True),
    ((17, 2), (0, 0), 7, 7, 128, 128, False, (16, 24, 24), "qk", False, True),
    ((40,), (100,), 16, 1, 128, 64, False, (0, 32, 0), "k", True, True),
    ((3, 70), (9, 1), 5, 5, 256, 256, True, (100, 28), "q", True, False),
    ((6,), (0,), 2, 2, 256, 16, False, None, "qk", False, True),
    ((9, 4), (3, 0), 3, 1, 128, 0, False, None, "qk", True, True),
    ((700, 300), (0, 20), 8, 2, 64, 64, True, None, "qk", True, True),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rotate(case, dtype):
    rows, history, hq, hkv, d, rot, mixed, sections, norms, store, k_out = CASES[case]
    gen = torch.Generator().manual_seed(100 + case)
    dt, pad, before = DT[dtype], 3, 2
    total = before + sum(rows) + pad
    lens = [h + n for h, n in zip(history, rows)]
    pool = Pool(lens, 16 if case % 2 else 32, hkv, d, dtype, gen, head_major=case % 3 == 1)
    qkv = (4 * torch.randn(total, hq + 2 * hkv, d, generator=gen)).to(dt).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    weights = [torch.randn(d, generator=gen).to(dt).cuda() if x in norms else None for x in "qk"]
    table = table_of(400 if sections else max(lens) + 1, rot) if rot else None
    axes = len(sections) if sections else 1
    positions = torch.randint(0, 400, (axes, total), generator=gen).to(torch.int32).cuda() if sections else None
    p = pool.params(hq)
    stride = qkv.stride(0)
    r = ops.make_rows(total, max(rows), q_stride=stride, k_stride=stride, v_stride=stride)
    rope = ops.make_rope(rot, table_rows=0 if table is None else table.shape[0], interleaved=mixed, eps=EPS, sections=sections,
                         q_out_stride=hq * d + 64, k_out_stride=hkv * d + 8 * 16)
    q_out = torch.full((total, hq * d + 64), 7.0, dtype=dt, device="cuda")
    k_to = torch.full((total, hkv * d + 128), 7.0, dtype=dt, device="cuda") if k_out else None
    views = [None if x is None else x[:, :h * d].unflatten(1, (h, d)) for x, h in ((q_out, hq), (k_to, hkv))]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = [x.clone() for x in (pool.k, pool.v)]
    starts = cu(rows) + before
    ops.rotate(p, r, rope, q, k, starts, table, v=v if store else None, positions=positions, context_lens=pool.context,
               q_weight=weights[0], k_weight=weights[1], q_out=views[0], k_out=views[1], dev_status=status,
               **(dict(k_cache=pool.k, v_cache=pool.v, block_tables=pool.tables) if store else {}))
    assert int(status) == 0
    axis = [i for i, n in enumerate(sections) for _ in range(n)] if sections else [0] * (rot // 2)
    pos = torch.zeros(total, rot // 2, dtype=torch.long, device="cuda")
    at = before
    places = []
    for s, n in enumerate(rows):
        places.append(torch.arange(lens[s] - n, lens[s], device="cuda"))
        for i in range(rot // 2):
            pos[at:at + n, i] = positions[axis[i], at:at + n].long() if sections else places[s]
        at += n
    mine = slice(before, before + sum(rows))
    want_q = turned(q[mine], weights[0], rot, mixed, table, pos[mine])
    want_k = turned(k[mine], weights[1], rot, mixed, table, pos[mine])
    assert_close(views[0][mine], *want_q, "q")
    if k_out:
        assert_close(views[1][mine], *want_k, "k")
    for x, width in ((q_out, hq * d), (k_to, hkv * d)):  # rows of no sequence and what lies between rows
        if x is not None:
            assert (x[:before] == 7).all() and (x[before + sum(rows):] == 7).all() and (x[:, width:] == 7).all()
    at = 0
    mask = torch.zeros(pool.kv[0].shape[:2], dtype=torch.bool, device="cuda")
    for s, n in enumerate(rows if store else ()):
        page, slot = pool.tables[s].long()[places[s] // pool.page], places[s] % pool.page
        assert_close(pool.kv[0][page, slot], want_k[0][at:at + n], want_k[1][at:at + n], "stored k") if n else None
        assert torch.equal(pool.kv[1][page, slot], v[mine][at:at + n])
        mask[page, slot] = True
        at += n
    for now, was in zip((pool.k, pool.v), old):  # nothing else in the pool changed
        now, was = (x.transpose(1, 2) if case % 3 == 1 else x for x in (now, was))
        assert torch.equal(now[~mask].nan_to_num(5.0), was[~mask].nan_to_num(5.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_over_its_input_and_made_outputs(dtype):
    gen = torch.Generator().manual_seed(5)
    rows, hq, hkv, d = [11, 3], 6, 2, 128
    q, k = (torch.randn(14, h, d, generator=gen).to(DT[dtype]).cuda() for h in (hq, hkv))
    p = ops.prompt_params(num_seqs=2, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=dtype)
    r, table = ops.make_rows(14, 11), table_of(40, d)
    rope = ops.make_rope(d, table_rows=40, eps=EPS)
    lens = torch.tensor([30, 3], dtype=torch.int32, device="cuda")
    w = torch.randn(d, generator=gen).to(DT[dtype]).cuda()
    a, b = ops.rotate(p, r, rope, q, k, cu(rows), table, context_lens=lens, q_weight=w, k_weight=w)
    q2, k2 = q.clone(), k.clone()
    ops.rotate(p, r, rope, q2, k2, cu(rows), table, context_lens=lens, q_weight=w, k_weight=w, q_out=q2, k_out=k2)
    assert torch.equal(a, q2) and torch.equal(b, k2)


def test_refused_rows_are_left_out():
    gen = torch.Generator().manual_seed(6)
    rows, hq, hkv, d = [2, 2, 2, 2], 4, 2, 64
    pool = Pool([40, 20, 20, 20], 16, hkv, d, "bf16", gen)
    q, k, v = (torch.randn(8, h, d, generator=gen).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv))
    p, r, table = pool.params(hq), ops.make_rows(8, 2), table_of(39, d)
    rope = ops.make_rope(d, table_rows=39)
    context = torch.tensor([40, 1, 10000, 20], dtype=torch.int32, device="cuda")
    pool.tables[3, 1] = pool.pages
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    old = pool.k.clone()
    ops.rotate(p, r, rope, q, k, cu(rows), table, v=v, context_lens=context, q_out=q_out, k_out=k_out, k_cache=pool.k, v_cache=pool.v,
               block_tables=pool.tables, dev_status=status)
    assert int(status) == ops.PA_DEV_BAD_INDEX | ops.PA_DEV_BAD_LEN | ops.PA_DEV_BAD_PAGE
    # sequence 0: position 38 is in the table, 39 is not; 1 and 2: lengths; 3: no page, but the rows themselves are turned
    left = [int(i) for i in ((q_out == 7).flatten(1).all(1)).nonzero()]
    assert left == [1, 2, 3, 4, 5] and [int(i) for i in ((k_out == 7).flatten(1).all(1)).nonzero()] == left
    changed = (pool.k.nan_to_num(5.0) != old.nan_to_num(5.0)).flatten(2).any(2)
    assert int(changed.sum()) == 1 and bool(changed[pool.tables[0, 2].long(), 38 - 32])


def test_captured_and_replayed_with_far_pages():
    """One captured call for other rows, lengths and tables; pages whose offsets, in elements, pass 32 bits."""
    gen = torch.Generator().manual_seed(8)
    pages, page, hq, hkv, d, stride = 36, 16, 4, 2, 64, 1 << 26
    k_cache, v_cache = (torch.zeros(pages * stride, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p = ops.make_params(num_seqs=40, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page, num_pages=pages, max_blocks_per_seq=2,
                        max_context_len=32, dtype="bf16", strides=(stride, 0, 0))
    rope, table = ops.make_rope(d, table_rows=32, eps=EPS), table_of(32, d)
    total = 60
    q, k, v = (torch.randn(total, h, d, generator=gen).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv))
    r = ops.make_rows(total, 20)
    starts, lens, tables = cu([1] * 40), torch.zeros(40, dtype=torch.int32, device="cuda"), torch.full((40, 2), -1, dtype=torch.int32, device="cuda")
    q_out = torch.zeros_like(q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            ops.rotate(p, r, rope, q, k, starts, table, v=v, context_lens=lens, q_out=q_out, k_cache=k_cache, v_cache=v_cache, block_tables=tables)
    views = [x.as_strided((pages, page, hkv, d), (stride, hkv * d, d, 1)) for x in (k_cache, v_cache)]
    for counts in ([1] * 30 + [0] * 10, [0] * 35 + [20, 0, 3, 1, 2]):
        held = [n + (i % 9 if n else 0) for i, n in enumerate(counts)]
        starts.copy_(cu(counts))
        lens.copy_(torch.tensor(held, dtype=torch.int32))
        order = torch.randperm(pages, generator=gen).tolist()
        rows = [[order.pop() if b * page < L else -1 for b in range(2)] for L in held]
        tables.copy_(torch.tensor(rows, dtype=torch.int32))
        q_out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for s, (n, L) in enumerate(zip(counts, held)):
            if n:
                spot = torch.arange(L - n, L, device="cuda")
                pos = spot[:, None].expand(-1, d // 2)
                pg = tables[s].long()[spot // page]
                assert_close(q_out[at:at + n], *turned(q[at:at + n], None, d, False, table, pos), "q")
                assert_close(views[0][pg, spot % page], *turned(k[at:at + n], None, d, False, table, pos), "k")
                assert torch.equal(views[1][pg, spot % page], v[at:at + n])
            at += n
        assert (q_out[at:] == 7).all()
