"""Tokens behind an eviction: the kept keys have the positions that they were turned at, so a sequence's next rows are
turned at positions of their own count, which the caller passes, and stored at the shorter length."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import DT, assert_close, attend, bound, cu
from test_step_rotate import EPS, table_of, turned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_loop_with_a_budget(dtype):
    gen = torch.Generator().manual_seed(90)
    hq, hkv, d, page, pages, blocks = 8, 2, 64, 16, 40, 8
    dt, n, budget = DT[dtype], 2, 40
    prompts, scale = [60, 33], 1 / math.sqrt(d)
    p = ops.make_params(num_seqs=n, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page, num_pages=pages, max_blocks_per_seq=blocks,
                        max_context_len=blocks * page, dtype=dtype, out_dtype="f32")

    def rand(*shape):
        return torch.randn(shape, generator=gen).to(dt).cuda()

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    k_cache, v_cache = (torch.full((pages, page, hkv, d), math.nan, dtype=dt, device="cuda") for _ in range(2))
    ref, tables, lens, pairs = ints([0] * pages), torch.full((n, blocks), -1, dtype=torch.int32, device="cuda"), ints([0] * n), ints([[-1, -1]] * n)
    ws, status = torch.empty(ops.pages_workspace_size(p), dtype=torch.uint8, device="cuda"), ints([0])
    table, rope = table_of(200, d), ops.make_rope(d, table_rows=200, eps=EPS)
    gathered = torch.zeros(n, hkv, blocks * page, device="cuda")
    keys = [[None] * hkv for _ in range(n)]  # K and V of the keys that are there, in their order
    count = [0] * n                          # tokens so far: the next position

    def step(rows):
        """New rows of each sequence: turned and stored at their positions; their attention gathered; the budget kept."""
        total, most, starts = sum(rows), max(rows), cu(rows)
        q, k, v = rand(total, hq, d), rand(total, hkv, d), rand(total, hkv, d)
        places = [torch.arange(c, c + m) for c, m in zip(count, rows)]
        positions = torch.cat(places).to(torch.int32).cuda()
        ops.pages_resize(p, ref, tables, lens, ints([L + m for L, m in zip(lens.tolist(), rows)]), pairs, ws, dev_status=status)
        r = ops.make_rows(total, most)
        q1, k1 = ops.rotate(p, r, rope, q, k, starts, table, v=v, positions=positions, context_lens=lens, k_out=torch.empty_like(k), k_cache=k_cache,
                            v_cache=v_cache, block_tables=tables, dev_status=status)
        pos = positions.long()[:, None].expand(-1, d // 2)
        assert_close(q1, *turned(q, None, d, False, table, pos), "q")
        assert_close(k1, *turned(k, None, d, False, table, pos), "k")
        ops.key_weights(p, r, q1, starts, k_cache, tables, lens, gathered, decay=0.5, dev_status=status)
        at = 0
        for s, m in enumerate(rows):
            count[s] += m
            for g in range(hkv):
                new = (k1[at:at + m, g].clone(), v[at:at + m, g].clone())
                keys[s][g] = new if keys[s][g] is None else tuple(torch.cat([a, b]) for a, b in zip(keys[s][g], new))
            at += m
        weights, kept, cut = ops.evict(p, k_cache, v_cache, tables, lens, gathered, ints([budget] * n), first=2, recent=8, refcounts=ref, dev_status=status)
        ops.pages_resize(p, ref, tables, lens, cut, pairs, ws, dev_status=status)
        gathered.copy_(weights)
        for s in range(n):
            for g in range(hkv):
                keys[s][g] = tuple(x[kept[s, g, :int(lens[s])].long()] for x in keys[s][g])
        return q1, starts

    step(prompts)
    assert lens.tolist() == [40, 33]
    for i in range(12):
        q1, starts = step([1, 1])
        assert lens.tolist() == [40, min(40, 34 + i)] and count == [61 + i, 34 + i]
        out = ops.decode(p, q1, k_cache, v_cache, tables, lens, dev_status=status)
        for s in range(n):
            for h in range(hq):
                kk, vv = (x.double() for x in keys[s][h // (hq // hkv)])
                qq = q1[s:s + 1, h].double()
                o, w = attend(qq, kk, vv, torch.ones(1, len(kk), dtype=torch.bool, device="cuda"), scale)
                assert_close(out[s:s + 1, h], o, bound(o, w, qq, kk, scale, len(kk), dtype, "f32"), f"token {i} {s} {h}")
    assert int(status) == 0 and int((ref > 0).sum()) == 6
