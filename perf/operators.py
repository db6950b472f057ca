"""What is timed of the serving-step operators: attention of whole prompts, attention of a draft tree over the paged
cache, storing K/V rows into the pages, and the page operations (resize, fork, compact, copy).

``own`` false computes each in elementary torch operations; true calls the package's entry points.  Both work on the
same state.  Shapes come from the package's workloads (12/3 heads at head_dim 64, 28/4, 40/8, 32/8 and 64/8 at 128,
pages of 16 and 32) or are generic.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
RAGGED = "1,31,32,33,1771,3398,2264,1130,3732,409,2930,1214,777,2873,65,2500"  # around a page, then short to long


def listed():
    def attn(op, name, lens, dtype, hq, hkv, d, **kw):
        return dict(name=name, op=op, lens=lens, dtype=dtype, hq=hq, hkv=hkv, d=d, **kw)

    return [
        # four short chat turns of a small fp32 model: latency counts
        attn("prompt", "prompt_f32_short", "33,16,1,57", "f32", 12, 3, 64, pad=0),
        # one prompt of a 7B-shaped model, an odd length
        attn("prompt", "prompt_f16_one", "1641", "f16", 28, 4, 128, pad=0),
        # a batch of prompts as they arrive together, packed, with padding rows behind them
        attn("prompt", "prompt_bf16_ragged", "2560,130,1999,37,1024,511,2048,1,700,1300,256,1777", "bf16", 32, 8, 128, pad=13),
        # one long document
        attn("prompt", "prompt_bf16_long", "8192", "bf16", 64, 8, 128, pad=0),
        # seven drafts of a small fp32 model
        attn("tree", "tree_f32_small", "1024", "f32", 12, 3, 64, drafts="7", page=16),
        # sixteen drafts behind one chat of a 14B-shaped model: latency counts
        attn("tree", "tree_f16_one", "3254", "f16", 40, 8, 128, drafts="16", page=32),
        # a ragged batch, each request with a tree of its own size (none for two of them)
        attn("tree", "tree_bf16_ragged", RAGGED, "bf16", 32, 8, 128, drafts="26,7,64,1,13,40,0,26,33,8,60,26,0,17,5,48", page=32),
        # long contexts, full trees of 64
        attn("tree", "tree_bf16_long", "16384,15000,16000,12345,16383,9999,16384,14000", "bf16", 64, 8, 128,
             drafts="64,64,64,64,64,64,64,64", page=32),
        # the accepted drafts of a verified step, chosen by index
        attn("store", "store_accepted", RAGGED, "bf16", 32, 8, 128, rows="1,3,6,1,2,4,0,5,3,1,1,2,0,3,1,6", page=32, pick=True),
        # the K/V of a batch of whole prompts
        attn("store", "store_prompts", "8192,4096,1777,2560,37,5000,1,2111", "bf16", 64, 8, 128,
             rows="8192,4096,1777,2560,37,5000,1,2111", page=32, pick=False),
        # a beam step: each of 16 requests forks its best beam three times, all grow by a token, the losers go
        dict(name="pages_beam", op="beam", groups=16, width=4, low=700, high=2100, page=32, hkv=8, d=128, dtype="bf16", pages=4096),
        # requests come and go: half of them end, the pool is compacted, new ones take their pages; then the other half
        dict(name="pages_churn", op="churn", seqs=96, low=100, high=3000, page=32, hkv=8, d=128, dtype="bf16", pages=8192),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "tree", "tree", "tree", "store", "beam", "churn"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while hkv * group > 64:
        group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    d = rng.choice([64, 128, 128])
    c = dict(op=op, dtype=dtype, hkv=hkv, d=d)
    if op in ("prompt", "tree", "store"):
        c["hq"] = hkv * group
    if op == "prompt":
        n = _log(rng, 1, 12)
        top = 2500 if dtype != "f32" else 1200
        c["lens"] = ",".join(str(_log(rng, 1, top)) for _ in range(n))
        c["pad"] = rng.choice([0, 0, 3, 64])
        return c
    c["page"] = rng.choice([16, 32])
    if op == "tree":
        n = _log(rng, 1, 16)
        c["lens"] = ",".join(str(rng.choice([0, _log(rng, 1, 6000), _log(rng, 1, 6000), _log(rng, 1, 6000)])) for _ in range(n))
        c["drafts"] = ",".join(str(_log(rng, 1, 128)) for _ in range(n))
    elif op == "store":
        n = _log(rng, 1, 24)
        rows = [_log(rng, 1, 1500) for _ in range(n)]
        c["lens"] = ",".join(str(r + rng.choice([0, _log(rng, 1, 3000)])) for r in rows)
        c["rows"] = ",".join(map(str, rows))
        c["pick"] = rng.random() < 0.5
    elif op == "beam":
        c.update(groups=_log(rng, 1, 24), width=rng.randint(2, 4), low=_log(rng, 1, 400), high=0, pages=4096)
        c["high"] = c["low"] + _log(rng, 1, 1400)
    else:
        c.update(seqs=2 * _log(rng, 2, 48), low=_log(rng, 1, 200), high=0, pages=_log(rng, 8000, 40000))
        c["high"] = c["low"] + _log(rng, 1, 2500)
        c["hkv"] = min(c["hkv"], 4)
    return c


def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _spread(low, high, n):
    """n lengths in [low, high], fixed by their place."""
    return [low + (i * 7919 + 13) % (high - low + 1) for i in range(n)]


def _cu(rows, dev="cuda"):
    return torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device=dev)


def _tables(counts, pages, gen, shuffle_in=None):
    """Block tables of sequences with `counts` pages each, disjoint, in shuffled pages of the pool (or of its first part)."""
    total = sum(counts)
    order = torch.randperm(shuffle_in or pages, generator=gen, device="cuda").to(torch.int32)[:total]
    table = torch.full((len(counts), max(max(counts), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(counts):
        table[s, :n] = order[at:at + n]
        at += n
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, hkv, d = DT[case["dtype"]], case["hkv"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    s = {"case": case, "op": case["op"]}
    if case["op"] == "prompt":
        lens = _ints(case["lens"])
        total = sum(lens) + case["pad"]
        s.update(lens=lens, total=total, cu=_cu(lens), q=normal(total, case["hq"], d), k=normal(total, hkv, d), v=normal(total, hkv, d),
                 out=torch.zeros(total, case["hq"], d, dtype=dt, device="cuda"))
    elif case["op"] in ("tree", "store"):
        lens, page = _ints(case["lens"]), case["page"]
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 7
        s.update(lens=lens, pages=pages, tables=_tables(counts, pages, gen), context=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 k_cache=normal(pages, page, hkv, d), v_cache=normal(pages, page, hkv, d))
        if case["op"] == "tree":
            drafts = _ints(case["drafts"])
            total, most = sum(drafts), max(drafts)
            s.update(drafts=drafts, total=total, cu=_cu(drafts), words=-(-most // 32), q=normal(total, case["hq"], d), k=normal(total, hkv, d),
                     v=normal(total, hkv, d), out=torch.zeros(total, case["hq"], d, dtype=dt, device="cuda"))
            s["mask"] = _trees(drafts, s["words"], gen)
        else:
            rows = _ints(case["rows"])
            total = sum(rows)
            sources = total + (500 if case["pick"] else 0)
            s.update(rows=rows, total=total, sources=sources, cu=_cu(rows), k=normal(sources, hkv, d), v=normal(sources, hkv, d))
            s["index"] = torch.randperm(sources, generator=gen, device="cuda")[:total].to(torch.int32) if case["pick"] else None
    else:
        _prepare_pages(case, s, gen, normal)
    if own:
        _prepare_own(case, s)
    return s


def _trees(drafts, words, gen):
    """Ancestor masks of random trees: a draft sees itself and what its parent, an earlier draft, sees."""
    total = sum(drafts)
    pick = torch.rand(max(total, 1), generator=gen, device="cuda").cpu().tolist()
    rows, at = [], 0
    for n in drafts:
        seen = []
        for t in range(n):
            parent = int(pick[at + t] * t) if t else -1
            bits = (seen[parent] if t else 0) | (1 << t)
            seen.append(bits)
            rows.append([(bits >> (32 * w)) & 0xFFFFFFFF for w in range(words)])
        at += n
    wide = torch.tensor(rows, dtype=torch.int64).reshape(total, words)
    return torch.where(wide >= 1 << 31, wide - (1 << 32), wide).to(torch.int32).cuda()


def _prepare_pages(case, s, gen, normal):
    page, pages = case["page"], case["pages"]
    if case["op"] == "beam":
        groups, width = case["groups"], case["width"]
        lens = _spread(case["low"], case["high"], groups)
        counts = [-(-n // page) for n in lens]
        n = groups * width
        most = max(-(-(case["high"] + 1) // page), 1)
        table = torch.full((n, most), -1, dtype=torch.int32, device="cuda")
        first = _tables(counts, pages, gen, shuffle_in=sum(counts) + 50)
        table[:groups, :first.shape[1]] = first
        context = torch.zeros(n, dtype=torch.int32, device="cuda")
        context[:groups] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        src = torch.arange(groups, dtype=torch.int32, device="cuda").repeat(width - 1)
        s.update(src=src, dst=torch.arange(groups, n, dtype=torch.int32, device="cuda"))
        base = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s.update(grow=(base + 1).repeat(width), drop=torch.cat([base, torch.zeros(n - groups, dtype=torch.int32, device="cuda")]))
        used = first[first >= 0].long()
    else:
        n = case["seqs"]
        lens = _spread(case["low"], case["high"], n)
        counts = [-(-x // page) for x in lens]
        half = n // 2
        # the first half in the low pages, the second above them: what a pass leaves behind it
        low, high = sum(counts[:half]), sum(counts[half:])
        assert low + high <= pages
        a = _tables(counts[:half], low, gen)
        b = _tables(counts[half:], high, gen)
        most = max(counts)
        table = torch.full((n, most), -1, dtype=torch.int32, device="cuda")
        table[:half, :a.shape[1]] = a
        table[half:, :b.shape[1]] = torch.where(b >= 0, b + low, b)
        context = torch.tensor(lens, dtype=torch.int32, device="cuda")
        keep = torch.full((half,), -1, dtype=torch.int32, device="cuda")
        none = torch.zeros(half, dtype=torch.int32, device="cuda")
        s.update(end=[torch.cat([none, keep]), torch.cat([keep, none])],
                 begin=[torch.cat([context[:half], keep]), torch.cat([keep, context[half:]])])
        s["moves"] = [torch.full((pages, 2), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
        s["count"] = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
        used = torch.arange(low + high, device="cuda")
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    ref[used] = 1
    s.update(seqs=n, tables=table, context=context, ref=ref, pairs=torch.full((n, 2), -1, dtype=torch.int32, device="cuda"),
             k_cache=normal(pages, page, case["hkv"], case["d"]), v_cache=normal(pages, page, case["hkv"], case["d"]))


def _prepare_own(case, s):
    """The parameter blocks and workspaces that a user's program keeps."""
    from paged_kv_gqa_02_gb300 import ops
    heads = dict(num_q_heads=case.get("hq", case["hkv"]), num_kv_heads=case["hkv"], head_dim=case["d"], dtype=case["dtype"])
    if case["op"] == "prompt":
        s["p"] = ops.prompt_params(num_seqs=len(s["lens"]), out_dtype=case["dtype"], **heads)
        s["r"] = ops.make_rows(s["total"], max(s["lens"]))
        return
    blocks = s["tables"].shape[1]
    pages = s["k_cache"].shape[0]
    s["p"] = ops.make_params(num_seqs=s["tables"].shape[0], page_size=case["page"], num_pages=pages, max_blocks_per_seq=blocks,
                             max_context_len=blocks * case["page"], out_dtype=case["dtype"], **heads)
    if case["op"] == "tree":
        s["r"] = ops.make_rows(s["total"], max(s["drafts"]))
        n = ops.tree_workspace_size(s["p"], s["r"])
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    elif case["op"] == "store":
        s["r"] = ops.make_rows(s["total"], max(s["rows"]), source_rows=s["sources"])
    else:
        s["ws"] = torch.empty(ops.pages_workspace_size(s["p"]), dtype=torch.uint8, device="cuda")


def run(state):
    return (_run_own if own else _run_plain)(state)


# ---- the package's entry points ---------------------------------------------------------------------------------

def _run_own(s):
    from paged_kv_gqa_02_gb300 import ops
    if s["op"] == "prompt":
        return ops.prompt(s["p"], s["r"], s["q"], s["k"], s["v"], s["cu"], out=s["out"])
    if s["op"] == "tree":
        return ops.tree(s["p"], s["r"], s["q"], s["k"], s["v"], s["cu"], s["mask"], s["k_cache"], s["v_cache"], s["tables"],
                        s["context"], out=s["out"], workspace=s["ws"])
    if s["op"] == "store":
        ops.store(s["p"], s["r"], s["k"], s["v"], s["cu"], s["k_cache"], s["v_cache"], s["tables"], s["context"], row_index=s["index"])
        return {"k": s["k_cache"], "v": s["v_cache"]}
    p, ref, tables, context, ws = s["p"], s["ref"], s["tables"], s["context"], s["ws"]
    if s["op"] == "beam":
        ops.pages_fork(p, ref, tables, context, s["src"], s["dst"])
        ops.pages_resize(p, ref, tables, context, s["grow"], s["pairs"], ws)
        ops.pages_copy(p, s["k_cache"], s["v_cache"], s["pairs"])
        made = s["pairs"].clone()
        ops.pages_resize(p, ref, tables, context, s["drop"], s["pairs"], ws)
        return _pages_out(s, made)
    for i in range(2):
        ops.pages_resize(p, ref, tables, context, s["end"][i], s["pairs"], ws)
        ops.pages_compact(p, ref, tables, context, s["moves"][i], s["count"][i], ws)
        ops.pages_copy(p, s["k_cache"], s["v_cache"], s["moves"][i])
        ops.pages_resize(p, ref, tables, context, s["begin"][i], s["pairs"], ws)
    return _pages_out(s, s["pairs"])


def _pages_out(s, made):
    out = {"ref": s["ref"], "tables": s["tables"], "context": s["context"], "pairs": made, "k": s["k_cache"], "v": s["v_cache"]}
    if s["op"] == "churn":
        out.update(moves=list(s["moves"]), count=list(s["count"]))
    return out


# ---- the plain forms ----------------------------------------------------------------------------------------------

def _places(cu, total):
    """The sequence and the place in it of each packed row; rows behind the last sequence count as its last row."""
    n = cu.numel() - 1
    row = torch.minimum(torch.arange(total, device=cu.device, dtype=cu.dtype), cu[n] - 1)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return seq, (row - cu[seq]).long(), torch.arange(total, device=cu.device) < cu[n]


def _padded(x, cu, most):
    """Packed rows as [sequences, most, ...]; places past a sequence's end repeat some row of the tensor."""
    at = cu[:-1, None].long() + torch.arange(most, device=x.device)[None]
    return x[at.clamp(max=x.shape[0] - 1)]


def _softmax_v(q, k, v, see, scale):
    """softmax(scale q.k) v over the keys that `see` shows, in 32 bits: q [B,T,Hq,D], k and v [B,J,Hkv,D], see [B,T,J].
    A row that sees nothing is zero."""
    b, t, hq, d = q.shape
    hkv = k.shape[2]
    q = q.float().reshape(b, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    scores = torch.matmul(q, k.float().permute(0, 2, 3, 1)).mul_(scale).reshape(b, hkv, hq // hkv, t, -1)
    scores.masked_fill_(~see[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = weights.sum(-1, keepdim=True)
    o = torch.matmul(weights.reshape(b, hkv, -1, weights.shape[-1]), v.float().permute(0, 2, 1, 3)).reshape(b, hkv, hq // hkv, t, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 3, 1, 2, 4).reshape(b, t, hq, d)


def _gathered(s):
    """Each sequence's cached rows, [sequences, longest, Hkv, D]."""
    table, page = s["tables"].long().clamp(min=0), s["case"]["page"]
    b, n = table.shape
    return tuple(c[table].reshape(b, n * page, c.shape[2], c.shape[3]) for c in (s["k_cache"], s["v_cache"]))


def _run_plain(s):
    case = s["case"]
    scale = 1.0 / math.sqrt(case["d"])
    if s["op"] == "prompt":
        most = max(s["lens"])
        seq, place, real = _places(s["cu"], s["total"])
        step = torch.arange(most, device="cuda")
        see = (step[None, :] <= step[:, None])[None].expand(len(s["lens"]), most, most)
        o = _softmax_v(*(_padded(s[x], s["cu"], most) for x in "qkv"), see, scale)
        return torch.where(real[:, None, None], o[seq, place], 0.0).to(s["q"].dtype)
    if s["op"] == "tree":
        most = max(s["drafts"])
        seq, place, _ = _places(s["cu"], s["total"])
        k, v = _gathered(s)
        step = torch.arange(most, device="cuda")
        bits = (s["mask"][:, step // 32] >> (step % 32).to(torch.int32)) & 1
        drafts = (s["cu"][1:] - s["cu"][:-1])[:, None, None]
        see_drafts = (_padded(bits, s["cu"], most) == 1) & (step[None, None] < drafts)
        see_cache = (torch.arange(k.shape[1], device="cuda")[None] < s["context"][:, None])[:, None].expand(-1, most, -1)
        k = torch.cat([k, _padded(s["k"], s["cu"], most)], 1)
        v = torch.cat([v, _padded(s["v"], s["cu"], most)], 1)
        o = _softmax_v(_padded(s["q"], s["cu"], most), k, v, torch.cat([see_cache, see_drafts], 2), scale)
        return o[seq, place].to(s["q"].dtype)
    if s["op"] == "store":
        seq, place, _ = _places(s["cu"], s["total"])
        at = (s["context"][seq] - (s["cu"][1:] - s["cu"][:-1])[seq]).long() + place
        page = s["tables"][seq, at // case["page"]].long()
        k, v = (s[x] if s["index"] is None else s[x][s["index"].long()] for x in "kv")
        s["k_cache"][page, at % case["page"]] = k
        s["v_cache"][page, at % case["page"]] = v
        return {"k": s["k_cache"], "v": s["v_cache"]}
    if s["op"] == "beam":
        _plain_fork(s, s["src"].long(), s["dst"].long())
        made = _plain_resize(s, s["grow"])
        _plain_copy(s, made)
        _plain_resize(s, s["drop"])
        return _pages_out(s, made)
    _plain_half(s, 0)
    return _pages_out(s, _plain_half(s, 1))


def _plain_half(s, i):
    _plain_resize(s, s["end"][i])
    _plain_compact(s, s["moves"][i], s["count"][i])
    _plain_copy(s, s["moves"][i])
    return _plain_resize(s, s["begin"][i])


def _plain_fork(s, src, dst):
    table, context, page = s["tables"], s["context"], s["case"]["page"]
    used = torch.arange(table.shape[1], device="cuda")[None] < ((context[src] + page - 1) // page)[:, None]
    row = torch.where(used, table[src], table[dst])
    table[dst] = row
    context[dst] = context[src]
    s["ref"].index_add_(0, row.clamp(min=0).reshape(-1), used.reshape(-1).to(torch.int32))


def _free_order(free):
    """The k-th free page, for each k."""
    n = free.numel()
    rank = torch.where(free, free.cumsum(0) - 1, n)
    return torch.zeros(n + 1, dtype=torch.int64, device="cuda").scatter_(0, rank, torch.arange(n, device="cuda"))


def _plain_resize(s, new):
    table, context, ref, page = s["tables"], s["context"], s["ref"], s["case"]["page"]
    pages, blocks = ref.numel(), table.shape[1]
    asked = new >= 0
    n = torch.where(asked, new, context)
    had, has = (context + page - 1) // page, (n + page - 1) // page
    edge = torch.minimum(context, n)
    at = (edge // page).long().clamp(max=blocks - 1)[:, None]
    front = table.gather(1, at)[:, 0]
    copy = asked & (edge % page != 0) & (ref[front.clamp(min=0).long()] > 1)
    need = (has - had).clamp(min=0) + copy.to(torch.int32)
    last = need.cumsum(0)
    free = ref == 0
    ok = asked & ((need == 0) | (last <= free.sum()))
    copy = copy & ok
    order = _free_order(free)
    first = last - need
    fresh = torch.where(copy, order[first.clamp(max=pages)].to(torch.int32), -1)
    made = torch.stack([torch.where(copy, front, -1), fresh], 1)
    block = torch.arange(blocks, device="cuda")[None]
    grown = (block >= had[:, None]) & (block < has[:, None]) & ok[:, None]
    gone = (block >= has[:, None]) & (block < had[:, None]) & ok[:, None]
    taken = order[(first[:, None] + copy[:, None].to(torch.int64) + block - had[:, None]).clamp(0, pages)].to(torch.int32)
    change = torch.zeros(pages, dtype=torch.int32, device="cuda")
    change.index_add_(0, table.clamp(min=0).reshape(-1), -gone.reshape(-1).to(torch.int32))
    change.index_add_(0, front.clamp(min=0), -copy.to(torch.int32))
    change.index_add_(0, taken.reshape(-1), grown.reshape(-1).to(torch.int32))
    change.index_add_(0, fresh.clamp(min=0), copy.to(torch.int32))
    table.copy_(torch.where(grown, taken, torch.where(gone, -1, table)))
    table.scatter_(1, at, torch.where(copy[:, None], fresh[:, None], table.gather(1, at)))
    ref += change
    context.copy_(torch.where(ok, n, context))
    return made


def _plain_compact(s, moves, count):
    table, context, ref, page = s["tables"], s["context"], s["ref"], s["case"]["page"]
    pages = ref.numel()
    live = ref > 0
    kept = live.sum()
    at = torch.arange(pages, device="cuda")
    high = live & (at >= kept)
    rank = torch.where(high, high.cumsum(0) - 1, pages)
    hole = _free_order(~live)[rank.clamp(max=pages)]
    to = torch.where(high, hole, at)
    both = torch.stack([at, to], 1).to(torch.int32)
    room = torch.full((pages + 1, 2), -1, dtype=torch.int32, device="cuda")
    room.scatter_(0, rank[:, None].expand(-1, 2), both)
    moves.copy_(room[:pages])
    count.copy_(high.sum())
    old = ref.clone()
    ref.masked_fill_(high, 0)
    ref.index_add_(0, to, torch.where(high, old, 0))
    used = torch.arange(table.shape[1], device="cuda")[None] < ((context + page - 1) // page)[:, None]
    table.copy_(torch.where(used, to[table.clamp(min=0).long()].to(torch.int32), table))


def _plain_copy(s, pairs):
    src, dst = pairs[pairs[:, 0] >= 0].long().unbind(1)
    s["k_cache"][dst] = s["k_cache"][src]
    s["v_cache"][dst] = s["v_cache"][src]


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    e, hkv, d = SIZE[case["dtype"]], case["hkv"], case["d"]
    if case["op"] == "prompt":
        lens = _ints(case["lens"])
        return {"bytes": e * d * sum(lens) * (2 * case["hq"] + 2 * hkv), "flops": 4 * d * case["hq"] * sum(n * (n + 1) // 2 for n in lens)}
    if case["op"] == "tree":
        pairs = list(zip(_ints(case["lens"]), _ints(case["drafts"])))
        read = sum(n for n, t in pairs if t) + sum(t for _, t in pairs)
        return {"bytes": e * d * (2 * hkv * read + 2 * case["hq"] * sum(t for _, t in pairs)), "flops": 4 * d * case["hq"] * sum(t * (n + 1) for n, t in pairs)}
    if case["op"] == "store":
        return {"bytes": 4 * e * d * hkv * sum(_ints(case["rows"])), "flops": 0}
    page = case["page"]
    each = 4 * e * d * hkv * page  # K and V of a page, read and written
    if case["op"] == "beam":
        lens = _spread(case["low"], case["high"], case["groups"])
        copies = case["width"] * sum(1 for n in lens if n % page)
        return {"bytes": each * copies + 4 * case["pages"] + 8 * case["width"] * sum(-(-n // page) for n in lens), "flops": 0}
    counts = [-(-n // page) for n in _spread(case["low"], case["high"], case["seqs"])]
    half = case["seqs"] // 2
    moves = 2 * min(sum(counts[:half]), sum(counts[half:]))
    return {"bytes": each * moves + 2 * 4 * 2 * case["pages"] + 16 * sum(counts), "flops": 0}


# ---- the definitions in 64 bits, sequence by sequence ---------------------------------------------------------------

def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = was
    if case["op"] in ("prompt", "tree"):
        return _exact_attention(case, s)
    if case["op"] == "store":
        k, v, at = s["k_cache"].double(), s["v_cache"].double(), 0
        for i, n in enumerate(s["rows"]):
            for new, pool in ((s["k"], k), (s["v"], v)):
                rows = torch.arange(at, at + n, device="cuda") if s["index"] is None else s["index"][at:at + n].long()
                spot = torch.arange(s["lens"][i] - n, s["lens"][i], device="cuda")
                pool[s["tables"][i].long()[spot // case["page"]], spot % case["page"]] = new[rows].double()
            at += n
        return {"k": k, "v": v}
    return _exact_pages(case, s)


def _exact_attention(case, s):
    d, hq, group = case["d"], case["hq"], case["hq"] // case["hkv"]
    out = torch.zeros(s["total"], hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for i, n in enumerate(s["lens"] if case["op"] == "prompt" else s["drafts"]):
        rows = slice(at, at + n)
        at += n
        for h in range(hq if n else 0):
            g = h // group
            q, k, v = s["q"][rows, h].double(), s["k"][rows, g].double(), s["v"][rows, g].double()
            if case["op"] == "prompt":
                see = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
            else:
                pages = s["tables"][i, : -(-s["lens"][i] // case["page"])].long()
                k = torch.cat([s["k_cache"][pages, :, g].double().reshape(-1, d)[: s["lens"][i]], k])
                v = torch.cat([s["v_cache"][pages, :, g].double().reshape(-1, d)[: s["lens"][i]], v])
                word = s["mask"][rows].long()
                see = torch.stack([(word[:, j // 32] >> (j % 32)) & 1 for j in range(n)], 1) == 1
                see = torch.cat([torch.ones(n, s["lens"][i], dtype=torch.bool, device="cuda"), see], 1)
            weights = torch.softmax((q @ k.T / math.sqrt(d)).masked_fill(~see, -math.inf), -1).nan_to_num(0.0)
            out[rows, h] = weights @ v
    return out


def _exact_pages(case, s):
    """The pools after a pass, by a walk through the definition on the host."""
    page, pages, n = case["page"], case["pages"], s["seqs"]
    table, length, ref = s["tables"].tolist(), s["context"].tolist(), s["ref"].tolist()
    k, v = s["k_cache"].double(), s["v_cache"].double()

    def up(x):
        return -(-x // page)

    def copy(made):
        if made:
            a, b = (torch.tensor(x, device="cuda") for x in zip(*made))
            for pool in (k, v):
                pool[b] = pool[a]

    def resize(new):
        free, made, used, old = [i for i in range(pages) if ref[i] == 0], [], 0, list(ref)
        for i in range(n):
            if new[i] < 0:
                continue
            edge = min(length[i], new[i])
            shared = edge % page != 0 and old[table[i][edge // page]] > 1
            need = max(0, up(new[i]) - up(length[i])) + shared
            used += need
            if need and used > len(free):
                continue
            mine = free[used - need:used]
            if shared:
                to = mine.pop(0)
                made.append((table[i][edge // page], to))
                ref[table[i][edge // page]] -= 1
                ref[to] += 1
                table[i][edge // page] = to
            for b in range(up(new[i]), up(length[i])):
                ref[table[i][b]] -= 1
                table[i][b] = -1
            for b in range(up(length[i]), up(new[i])):
                table[i][b] = mine.pop(0)
                ref[table[i][b]] += 1
            length[i] = new[i]
        return made

    def compact():
        live = [i for i in range(pages) if ref[i] > 0]
        holes = [i for i in range(len(live)) if ref[i] == 0]
        to = dict(zip([i for i in live if i >= len(live)], holes))
        for a, b in to.items():
            ref[a], ref[b] = 0, ref[a]
        for i in range(n):
            for b in range(up(length[i])):
                table[i][b] = to.get(table[i][b], table[i][b])
        return list(to.items())

    if case["op"] == "beam":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            length[b] = length[a]
            for i in range(up(length[a])):
                table[b][i] = table[a][i]
                ref[table[a][i]] += 1
        copy(resize(s["grow"].tolist()))
        resize(s["drop"].tolist())
    else:
        for i in range(2):
            resize(s["end"][i].tolist())
            copy(compact())
            resize(s["begin"][i].tolist())
    return {"k": k, "v": v}
