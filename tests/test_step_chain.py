"""The operators of a serving step one after another, as a program runs them: prompts in, drafts verified and stored, keys
weighed and evicted, a token decoded over what is left."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import DT, assert_close, attend, bound, cu
from test_step_rotate import EPS, table_of, turned
from test_step_verify import walk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_step(dtype):
    gen = torch.Generator().manual_seed(40)
    hq, hkv, d, page, pages, blocks, vocab = 8, 2, 64, 16, 200, 20, 211
    dt, n = DT[dtype], 3
    prompts, drafts = [60, 17, 33], [5, 3, 4]
    scale = 1 / math.sqrt(d)
    p = ops.make_params(num_seqs=n, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page, num_pages=pages, max_blocks_per_seq=blocks,
                        max_context_len=blocks * page, dtype=dtype, out_dtype="f32")

    def rand(*shape):
        return torch.randn(shape, generator=gen).to(dt).cuda()

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    k_cache, v_cache = (torch.full((pages, page, hkv, d), math.nan, dtype=dt, device="cuda") for _ in range(2))
    ref, tables, lens, pairs = ints([0] * pages), torch.full((n, blocks), -1, dtype=torch.int32, device="cuda"), ints([0] * n), ints([[-1, -1]] * n)
    ws, status = torch.empty(ops.pages_workspace_size(p), dtype=torch.uint8, device="cuda"), ints([0])
    table, weight = table_of(blocks * page, d), rand(d)
    rope = ops.make_rope(d, table_rows=blocks * page, eps=EPS)
    gathered = torch.zeros(n, hkv, blocks * page, device="cuda")

    # the prompts: room, rotation with the store, what the keys gather
    total, starts = sum(prompts), cu(prompts)
    qkv = rand(total, hq + 2 * hkv, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    stride = qkv.stride(0)
    ops.pages_resize(p, ref, tables, lens, ints(prompts), pairs, ws, dev_status=status)
    r = ops.make_rows(total, max(prompts), q_stride=stride, k_stride=stride, v_stride=stride)
    q1, k1 = ops.rotate(p, r, rope, q, k, starts, table, v=v, context_lens=lens, q_weight=weight, k_weight=weight, k_out=torch.empty_like(k).contiguous(),
                        k_cache=k_cache, v_cache=v_cache, block_tables=tables, dev_status=status)
    flat = ops.make_rows(total, max(prompts), v_stride=stride)
    out = ops.prompt(p, flat, q1, k1, v, starts, dev_status=status)
    ops.key_weights(p, flat, q1, starts, k_cache, tables, lens, gathered, decay=0.0, dev_status=status)
    keys = [[(k1[a:a + m, g].clone(), v[a:a + m, g].clone()) for g in range(hkv)] for a, m in zip(starts.tolist(), prompts)]
    pos = torch.cat([torch.arange(m, device="cuda") for m in prompts])[:, None].expand(-1, d // 2)
    assert_close(q1, *turned(q, weight, d, False, table, pos), "q")
    assert_close(k1, *turned(k, weight, d, False, table, pos), "k")
    sums = gathered.sum(2).cpu()
    for s, m in enumerate(prompts):  # each row's weights add up to one
        assert torch.allclose(sums[s], torch.full((hkv,), float(m * hq // hkv)), rtol=1e-4)
    o, w = attend(q1[:60, 5].double(), keys[0][1][0].double(), keys[0][1][1].double(), torch.ones(60, 60, dtype=torch.bool, device="cuda").tril(), scale)
    assert_close(out[:60, 5], o, bound(o, w, q1[:60, 5].double(), keys[0][1][0].double(), scale, 60, dtype, "f32"), "prompt")

    # drafts: attention as a tree (a chain here), verification, room, the store of the accepted
    total, starts = sum(drafts), cu(drafts)
    q2, k2, v2 = rand(total, hq, d), rand(total, hkv, d), rand(total, hkv, d)
    mask = ints([(1 << (t + 1)) - 1 for m in drafts for t in range(m)]).reshape(total, 1)
    r = ops.make_rows(total, max(drafts))
    ops.tree(p, r, q2, k2, v2, starts, mask, k_cache, v_cache, tables, lens, dev_status=status)
    logits, draft = 2 * rand(total, vocab), 2 * rand(total, vocab)
    draft = (logits + 0.3 * draft).to(dt)
    parents = ints([max(t - 1, 0) for m in drafts for t in range(m)])
    tokens = draft.float().argmax(1).roll(1).to(torch.int32)
    uniform, noise, heat = torch.rand(total, generator=gen).cuda(), torch.empty(n, vocab).exponential_(generator=gen).cuda(), torch.ones(n, device="cuda")
    vp = ops.verify_params(num_seqs=n, dtype=dtype)
    accepted, ends, nexts, new_lens = ops.verify(vp, r, logits, draft, tokens, parents, starts, heat, uniform, noise, context_lens=lens, dev_status=status)
    at = 0
    paths = []
    for s, m in enumerate(drafts):
        path, token, margin = walk(logits[at:at + m], draft[at:at + m], tokens[at:at + m].tolist(), parents[at:at + m].tolist(), 1.0, uniform[at:at + m], noise[s])
        assert margin > 2.0 ** -16 and accepted[ends[s]:ends[s + 1]].tolist() == [at + t for t in path] and int(nexts[s]) == token
        paths.append([at + t for t in path])
        at += m
    ops.pages_resize(p, ref, tables, lens, new_lens, pairs, ws, dev_status=status)
    ops.pages_copy(p, k_cache, v_cache, pairs, dev_status=status)
    ops.store(p, r, k2, v2, ends, k_cache, v_cache, tables, lens, row_index=accepted, dev_status=status)
    one = ops.make_rows(n, 1)
    q3 = rand(n, hq, d)
    before = gathered.clone()
    ops.key_weights(p, one, q3, cu([1] * n), k_cache, tables, lens, gathered, dev_status=status)
    held = lens.tolist()
    assert held == [m + len(x) for m, x in zip(prompts, paths)]
    for s in range(n):
        for g in range(hkv):
            keys[s][g] = tuple(torch.cat([old, new[paths[s], g]]) for old, new in zip(keys[s][g], (k2, v2)))

    # eviction, once the longest is over its budget, and the pages back
    budget = [40, -1, 20]
    kept_weights, kept, cut = ops.evict(p, k_cache, v_cache, tables, lens, gathered, ints(budget), first=2, recent=8, refcounts=ref, dev_status=status)
    assert cut.tolist() == budget
    ops.pages_resize(p, ref, tables, lens, cut, pairs, ws, dev_status=status)
    assert lens.tolist() == [40, held[1], 20] and int((ref > 0).sum()) == 3 + -(-held[1] // page) + 2
    for s in range(n):
        for g in range(hkv):
            m = int(lens[s])
            index = kept[s, g, :m].long()
            assert index.tolist() == sorted(set(index.tolist())) and torch.equal(kept_weights[s, g, :m], gathered[s, g, index])
            if budget[s] >= 0:
                assert index[:2].tolist() == [0, 1] and index[-8:].tolist() == list(range(held[s] - 8, held[s]))
                rest = torch.ones(held[s], dtype=torch.bool, device="cuda")
                rest[index] = False
                assert float(gathered[s, g, :held[s]][rest].max()) <= float(gathered[s, g, index[2:-8]].min())
            keys[s][g] = tuple(x[index] for x in keys[s][g])

    # a token decoded over what is left
    q4 = rand(n, hq, d)
    out = ops.decode(p, q4, k_cache, v_cache, tables, lens, dev_status=status)
    for s in range(n):
        for h in range(hq):
            kk, vv = (x.double() for x in keys[s][h // (hq // hkv)])
            qq = q4[s:s + 1, h].double()
            o, w = attend(qq, kk, vv, torch.ones(1, len(kk), dtype=torch.bool, device="cuda"), scale)
            assert_close(out[s:s + 1, h], o, bound(o, w, qq, kk, scale, len(kk), dtype, "f32"), f"decode {s} {h}")
    assert int(status) == 0 and before.shape == gathered.shape
