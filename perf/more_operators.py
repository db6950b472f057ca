"""What is timed of the operators around the serving step's attention: norms and rotation of queries and keys with their
store into the pages, verification of drafted tokens, the attention weight that each cached key has gathered, and the
eviction of the keys that gathered least.

``own`` false computes each in elementary torch operations; true calls the package's entry points.  Both work on the
same state.  Heads, pages and lengths come from the package's workloads (12/3 heads at head_dim 64, 28/4, 40/8, 32/8
and 64/8 at 128, pages of 16 and 32); vocabularies are generic.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
RAGGED = "1,31,32,33,1771,3398,2264,1130,3732,409,2930,1214,777,2873,65,2500"  # around a page, then short to long
TREES = "26,7,64,1,13,40,1,26,33,8,60,26,2,17,5,48"  # rows of a request's tree, its certain token among them
EPS = 1e-6


def listed():
    def rotate(name, rows, lens, dtype, hq, hkv, d, rot, **kw):
        return dict(name=name, op="rotate", rows=rows, lens=lens, dtype=dtype, hq=hq, hkv=hkv, d=d, rot=rot, page=kw.pop("page", 32), pad=kw.pop("pad", 0),
                    sections=kw.pop("sections", ""), mixed=kw.pop("mixed", False), norm=kw.pop("norm", True), store=kw.pop("store", True), k_out=kw.pop("k_out", True))

    def verify(name, rows, vocab, dtype, draft, chain, greedy):
        return dict(name=name, op="verify", rows=rows, vocab=vocab, dtype=dtype, draft=draft, chain=chain, greedy=greedy)

    def weights(name, rows, lens, dtype, hq, hkv, d, page, decay):
        return dict(name=name, op="weights", rows=rows, lens=lens, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, decay=decay)

    def evict(name, lens, keep, first, recent, dtype, hkv, d, page):
        return dict(name=name, op="evict", lens=lens, keep=keep, first=first, recent=recent, dtype=dtype, hkv=hkv, d=d, page=page)

    return [
        # the next token of five chats of a small fp32 model, straight into the pages: latency counts
        rotate("rotate_f32_tokens", "1,1,1,1,1", "33,16,1,1024,257", "f32", 12, 3, 64, 64, page=16, norm=False, k_out=False),
        # a prompt of text and images of a 7B-shaped model: three axes of positions, no pages yet
        rotate("rotate_f16_axes", "1641", "1641", "f16", 28, 4, 128, 128, sections="16,24,24", store=False),
        # chunks of prompts as they arrive together, half of each head turning in neighbouring pairs, padding rows behind them
        rotate("rotate_bf16_ragged", "2560,130,1999,37,1024,511,2048,1,700,1300,256,1777", "2560,1130,1999,4037,1024,2511,2048,1,1700,1300,256,3777",
               "bf16", 32, 8, 128, 64, mixed=True, pad=13),
        # four long documents
        rotate("rotate_bf16_long", "8192,8192,8192,8000", "8192,8192,8192,8000", "bf16", 64, 8, 128, 128),
        # one chat, a chain of four drafts that were looked up in its own text (no draft distribution): latency counts
        verify("verify_f32_chain", "5", 32000, "f32", False, True, 0),
        # a batch of chats, chains of five, an odd vocabulary, some of them greedy
        verify("verify_f16_chains", ",".join(["6"] * 64), 50021, "f16", True, True, 5),
        # a ragged batch, each request with a tree of its own size
        verify("verify_bf16_trees", TREES, 131072, "bf16", True, False, 0),
        # the next token of one chat: latency counts
        weights("weights_f16_one", "1", "3254", "f16", 40, 8, 128, 32, 1.0),
        # the next token of long contexts, the old weights fading
        weights("weights_bf16_long", "1,1,1,1,1,1,1,1", "16384,15000,16000,12345,16383,9999,16384,14000", "bf16", 64, 8, 128, 32, 0.96875),
        # whole prompts, each key's weight over all rows
        weights("weights_bf16_prompts", "2560,130,1999,37", "2560,130,1999,37", "bf16", 32, 8, 128, 32, 1.0),
        # four short requests of a small fp32 model shed a few pages each
        evict("evict_f32_few", "300,257,290,64", "256,192,280,64", 4, 32, "f32", 3, 64, 16),
        # long prompts shrink to the budget that their answers are decoded with
        evict("evict_bf16_prompts", "16384,15000,16000,12345,16383,9999,16384,14000", "2048,2048,2048,2048,4096,2048,8192,2048", 4, 64, "bf16", 8, 128, 32),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def _text(values):
    return ",".join(map(str, values))


def draw(rng):
    op = rng.choice(["rotate", "verify", "weights", "weights", "evict"])
    c = dict(op=op, dtype=rng.choice(["f32", "f16", "bf16", "bf16"]))
    if op == "verify":
        n = _log(rng, 1, 32)
        chain = rng.random() < 0.5
        c.update(rows=_text(_log(rng, 1, 8 if chain else 64) for _ in range(n)), vocab=_log(rng, 500, 131072), draft=rng.random() < 0.6, chain=chain,
                 greedy=rng.choice([0, 0, 1, n]))
        return c
    hkv, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while hkv * group > 64:
        group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    c.update(hkv=hkv, d=d, page=rng.choice([16, 32]))
    if op == "evict":
        lens = [_log(rng, 1, 12000) for _ in range(_log(rng, 1, 12))]
        part = rng.choice([0.1, 0.5, 0.9, 1.1])
        c.update(lens=_text(lens), keep=_text(max(1, int(part * n)) for n in lens), first=rng.choice([0, 1, 4, 16]), recent=rng.choice([0, 1, 32, 100]))
        return c
    c["hq"] = hkv * group
    if op == "rotate":
        rows = [_log(rng, 1, 2000) for _ in range(_log(rng, 1, 24))]
        rot = rng.choice([d, d, d // 2, 16])
        axes = rng.choice([1, 1, 3])
        a = rng.randint(0, rot // 2)
        b = rng.randint(0, rot // 2 - a)
        store = rng.random() < 0.7
        c.update(rows=_text(rows), lens=_text(n + rng.choice([0, _log(rng, 1, 3000)]) for n in rows), rot=rot, sections="" if axes == 1 else _text([a, b, rot // 2 - a - b]),
                 mixed=rng.random() < 0.3, norm=rng.random() < 0.7, store=store, k_out=not store or rng.random() < 0.5, pad=rng.choice([0, 0, 3, 64]))
        return c
    if rng.random() < 0.5:  # single tokens, or a few
        rows = [rng.choice([1, 1, 1, 2, 5]) for _ in range(_log(rng, 1, 32))]
        lens = [n + rng.choice([0, _log(rng, 1, 12000)]) for n in rows]
    else:  # the last rows of a prompt, or all of it
        rows = [_log(rng, 1, 1200 if c["dtype"] != "f32" else 500) for _ in range(_log(rng, 1, 4))]
        lens = [n + rng.choice([0, _log(rng, 1, 2000)]) for n in rows]
    c.update(rows=_text(rows), lens=_text(lens), decay=rng.choice([0.0, 0.96875, 1.0]))
    return c


def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _cu(rows):
    return torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device="cuda")


def _tables(lens, page, gen):
    """Block tables of sequences with these lengths, disjoint, in shuffled pages, and the pool's pages."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 7
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(counts), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(counts):
        table[s, :n] = order[at:at + n]
        at += n
    return table, pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    {"rotate": _prepare_rotate, "verify": _prepare_verify, "weights": _prepare_weights, "evict": _prepare_evict}[case["op"]](case, s, gen)
    if own:
        _prepare_own(case, s)
    return s


def _normal(gen, dt, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)


def _uniform(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)


def _prepare_rotate(case, s, gen):
    dt, hq, hkv, d, rot = DT[case["dtype"]], case["hq"], case["hkv"], case["d"], case["rot"]
    rows, lens = _ints(case["rows"]), _ints(case["lens"])
    total = sum(rows) + case["pad"]
    # one projection's output: queries, keys and values of a row beside one another
    s["qkv"] = _normal(gen, dt, total, hq + 2 * hkv, d)
    s.update(rows=rows, lens=lens, total=total, cu=_cu(rows), q=s["qkv"][:, :hq], k=s["qkv"][:, hq:hq + hkv], v=s["qkv"][:, hq + hkv:],
             context=torch.tensor(lens, dtype=torch.int32, device="cuda"), q_out=torch.zeros(total, hq, d, dtype=dt, device="cuda"),
             k_out=torch.zeros(total, hkv, d, dtype=dt, device="cuda") if case["k_out"] else None, q_weight=None, k_weight=None, positions=None)
    if case["norm"]:
        s.update(q_weight=(1 + 0.1 * _normal(gen, torch.float32, d)).to(dt), k_weight=(1 + 0.1 * _normal(gen, torch.float32, d)).to(dt))
    far = max(lens) + 1
    if case["sections"]:
        # text counts on along all axes; a run of rows in the middle is an image of 32 patches a line
        t = torch.arange(total, device="cuda")
        image = (t > total // 4) & (t < total // 2)
        p = torch.clamp(t - total // 4, min=0)
        s["positions"] = torch.stack([torch.where(image, total // 4, t), torch.where(image, total // 4 + p // 32, t), torch.where(image, total // 4 + p % 32, t)]).to(torch.int32)
        far = int(max(far, total + 32))
    angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2))
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if case["store"]:
        s["tables"], s["pages"] = _tables(lens, case["page"], gen)
        s.update(k_cache=_normal(gen, dt, s["pages"], case["page"], hkv, d), v_cache=_normal(gen, dt, s["pages"], case["page"], hkv, d))


def _prepare_verify(case, s, gen):
    dt, vocab, rows = DT[case["dtype"]], case["vocab"], _ints(case["rows"])
    total, n = sum(rows), len(rows)
    target = _normal(gen, torch.float32, total, vocab).mul_(4)  # a few likely tokens, a long tail
    draft = (target * 0.95 + 0.5 * _normal(gen, torch.float32, total, vocab)).to(dt)
    s.update(rows=rows, total=total, vocab=vocab, cu=_cu(rows), logits=target.to(dt), draft=draft if case["draft"] else None)
    # the parent of a draft: the row before it in a chain, some earlier row in a tree
    pick, parents, parent_rows, at = _uniform(gen, total).tolist(), [], [], 0
    for m in rows:
        mine = [0] + [t - 1 if case["chain"] else int(pick[at + t] * t) for t in range(1, m)]
        parents += mine
        parent_rows += [at + p for p in mine]
        at += m
    s["parents"] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    # each draft is drawn from the draft distribution behind its parent
    race = _uniform(gen, total, vocab).clamp_(min=1e-9).log_().neg_()
    s["tokens"] = (draft[torch.tensor(parent_rows, device="cuda")].float() - race.log_()).argmax(1).to(torch.int32)
    temperature = 0.7 + 0.6 * _uniform(gen, n)
    temperature[:case["greedy"]] = 0
    s.update(temperature=temperature, uniform=_uniform(gen, total), noise=_uniform(gen, n, vocab).clamp_(min=1e-9).log_().neg_().clamp_(min=1e-9),
             context=torch.tensor([100 + 37 * i for i in range(n)], dtype=torch.int32, device="cuda"))
    s.update(accepted=torch.full((total,), -1, dtype=torch.int32, device="cuda"), accepted_cu=torch.zeros(n + 1, dtype=torch.int32, device="cuda"),
             next=torch.zeros(n, dtype=torch.int32, device="cuda"), new_lens=torch.zeros(n, dtype=torch.int32, device="cuda"))


def _prepare_weights(case, s, gen):
    dt, rows, lens, hkv, d = DT[case["dtype"]], _ints(case["rows"]), _ints(case["lens"]), case["hkv"], case["d"]
    s["tables"], s["pages"] = _tables(lens, case["page"], gen)
    s.update(rows=rows, lens=lens, total=sum(rows), cu=_cu(rows), context=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             q=_normal(gen, dt, sum(rows), case["hq"], d), k_cache=_normal(gen, dt, s["pages"], case["page"], hkv, d))
    # what a key has gathered before is of the size of what a row gives it now
    s["weights"] = _normal(gen, torch.float32, len(lens), hkv, s["tables"].shape[1] * case["page"]).mul_(2).exp_().mul_(0.001)


def _prepare_evict(case, s, gen):
    dt, lens, keep, hkv, d = DT[case["dtype"]], _ints(case["lens"]), _ints(case["keep"]), case["hkv"], case["d"]
    s["tables"], s["pages"] = _tables(lens, case["page"], gen)
    slots = s["tables"].shape[1] * case["page"]
    s.update(lens=lens, context=torch.tensor(lens, dtype=torch.int32, device="cuda"), keep=torch.tensor(keep, dtype=torch.int32, device="cuda"),
             k_cache=_normal(gen, dt, s["pages"], case["page"], hkv, d), v_cache=_normal(gen, dt, s["pages"], case["page"], hkv, d),
             # what keys gather: most little, a few much; some keys were never looked at
             weights=_normal(gen, torch.float32, len(lens), hkv, slots).mul_(2).exp_(), kept=torch.full((len(lens), hkv, slots), -1, dtype=torch.int32, device="cuda"),
             weights_out=torch.zeros(len(lens), hkv, slots, dtype=torch.float32, device="cuda"), new_lens=torch.zeros(len(lens), dtype=torch.int32, device="cuda"))
    s["weights"].masked_fill_(_uniform(gen, len(lens), hkv, slots) < 0.05, 0.0)
    s["refcounts"] = torch.zeros(s["pages"], dtype=torch.int32, device="cuda")
    s["refcounts"][s["tables"][s["tables"] >= 0].long()] = 1


def _prepare_own(case, s):
    """The parameter blocks and workspaces that a user's program keeps."""
    from paged_kv_gqa_02_gb300 import ops
    if case["op"] == "verify":
        s["p"] = ops.verify_params(num_seqs=len(s["rows"]), dtype=case["dtype"])
        s["r"] = ops.make_rows(s["total"], max(s["rows"]))
        return
    heads = dict(num_q_heads=case.get("hq", case["hkv"]), num_kv_heads=case["hkv"], head_dim=case["d"], dtype=case["dtype"])
    if "tables" in s:
        blocks = s["tables"].shape[1]
        s["p"] = ops.make_params(num_seqs=len(s["lens"]), page_size=case["page"], num_pages=s["pages"], max_blocks_per_seq=blocks,
                                 max_context_len=blocks * case["page"], out_dtype=case["dtype"], **heads)
    else:
        s["p"] = ops.prompt_params(num_seqs=len(s["lens"]), out_dtype=case["dtype"], **heads)
    if case["op"] == "rotate":
        stride = s["qkv"].stride(0)
        s["r"] = ops.make_rows(s["total"], max(s["rows"]), q_stride=stride, k_stride=stride, v_stride=stride)
        s["rope"] = ops.make_rope(case["rot"], table_rows=s["table"].shape[0], interleaved=case["mixed"], eps=EPS,
                                  sections=_ints(case["sections"]) if case["sections"] else None)
    elif case["op"] == "weights":
        s["r"] = ops.make_rows(s["total"], max(s["rows"]))
        s["ws"] = torch.empty(max(ops.key_weights_workspace_size(s["p"], s["r"]), 1), dtype=torch.uint8, device="cuda")


def run(state):
    return (_run_own if own else _run_plain)(state)


# ---- the package's entry points ---------------------------------------------------------------------------------

def _run_own(s):
    from paged_kv_gqa_02_gb300 import ops
    case = s["case"]
    if s["op"] == "rotate":
        store = dict(k_cache=s["k_cache"], v_cache=s["v_cache"], block_tables=s["tables"]) if case["store"] else {}
        ops.rotate(s["p"], s["r"], s["rope"], s["q"], s["k"], s["cu"], s["table"], v=s["v"] if case["store"] else None, positions=s["positions"],
                   context_lens=s["context"], q_weight=s["q_weight"], k_weight=s["k_weight"], q_out=s["q_out"], k_out=s["k_out"], **store)
        return _rotate_out(s)
    if s["op"] == "verify":
        ops.verify(s["p"], s["r"], s["logits"], s["draft"], s["tokens"], s["parents"], s["cu"], s["temperature"], s["uniform"], s["noise"],
                   context_lens=s["context"], accepted=s["accepted"], accepted_cu=s["accepted_cu"], next_tokens=s["next"], new_lens=s["new_lens"])
        return _verify_out(s)
    if s["op"] == "weights":
        ops.key_weights(s["p"], s["r"], s["q"], s["cu"], s["k_cache"], s["tables"], s["context"], s["weights"], decay=case["decay"], workspace=s["ws"])
        return s["weights"]
    ops.evict(s["p"], s["k_cache"], s["v_cache"], s["tables"], s["context"], s["weights"], s["keep"], s["weights_out"], s["kept"], s["new_lens"],
              first=case["first"], recent=case["recent"], refcounts=s["refcounts"])
    return _evict_out(s)


def _rotate_out(s):
    out = {"q": s["q_out"]}
    if s["case"]["k_out"]:
        out["k"] = s["k_out"]
    if s["case"]["store"]:
        out.update(k_cache=s["k_cache"], v_cache=s["v_cache"])
    return out


def _verify_out(s):
    return {x: s[x] for x in ("accepted", "accepted_cu", "next", "new_lens")}


def _evict_out(s):
    return {x: s[x] for x in ("k_cache", "v_cache", "weights_out", "kept", "new_lens")}


# ---- the plain forms ----------------------------------------------------------------------------------------------

def _run_plain(s):
    return {"rotate": _plain_rotate, "verify": _plain_verify, "weights": _plain_weights, "evict": _plain_evict}[s["op"]](s)


def _places(cu, total):
    """The sequence and the place in it of each packed row; rows behind the last sequence count as its last row."""
    n = cu.numel() - 1
    row = torch.minimum(torch.arange(total, device=cu.device, dtype=cu.dtype), cu[n] - 1)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return seq, (row - cu[seq]).long(), torch.arange(total, device=cu.device) < cu[n]


def _plain_rotate(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    seq, place, real = _places(s["cu"], s["total"])
    at = (s["context"][seq] - (s["cu"][1:] - s["cu"][:-1])[seq]).long() + place
    if s["positions"] is None:
        cs = s["table"][at]
        cos, sin = cs[:, None, :half], cs[:, None, half:]
    else:
        axis = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(_ints(case["sections"])).cuda(), output_size=half)
        pos, pair = s["positions"].long()[axis].T, torch.arange(half, device="cuda")[None]
        cos, sin = s["table"][pos, pair][:, None], s["table"][pos, half + pair][:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
        t = x[..., :rot]
        a, b = (t[..., 0::2], t[..., 1::2]) if case["mixed"] else (t[..., :half], t[..., half:])
        pair = [a * cos - b * sin, a * sin + b * cos]
        t = torch.stack(pair, -1).flatten(-2) if case["mixed"] else torch.cat(pair, -1)
        return torch.cat([t, x[..., rot:]], -1).to(s["q"].dtype)

    q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
    s["q_out"].copy_(torch.where(real[:, None, None], q, s["q_out"]))
    if case["k_out"]:
        s["k_out"].copy_(torch.where(real[:, None, None], k, s["k_out"]))
    if case["store"]:
        seq, at, n = seq[:sum(s["rows"])], at[:sum(s["rows"])], sum(s["rows"])
        page = s["tables"][seq, at // case["page"]].long()
        s["k_cache"][page, at % case["page"]] = k[:n]
        s["v_cache"][page, at % case["page"]] = s["v"][:n]
    return _rotate_out(s)


def _plain_verify(s):
    """All sequences at once, row by row: a row whose parent is the last accepted one is tried against what is left of
    the target's distribution behind it.  Rows come after their parents, so one pass over them walks the tree."""
    cu, n, vocab = s["cu"].long(), len(s["rows"]), s["vocab"]
    every = torch.arange(n, device="cuda")
    greedy = ~(s["temperature"] > 0)
    heat = torch.where(greedy, 1.0, s["temperature"]).double()[:, None]

    def soft(x):
        return torch.softmax(x.double() / heat, 1)

    def one_hot(token):
        return torch.arange(vocab, device="cuda")[None] == token[:, None]

    here = torch.zeros(n, dtype=torch.int64, device="cuda")  # the last accepted row, in its sequence
    rows = cu[1:] - cu[:-1]
    left = soft(s["logits"][cu[:-1]])
    best = s["logits"][cu[:-1]].max(1).indices
    draft = soft(s["draft"][cu[:-1]]) if s["draft"] is not None else None
    took = torch.zeros(s["total"], dtype=torch.bool, device="cuda")
    took[cu[:-1]] = True
    for t in range(1, max(s["rows"])):
        row = (cu[:-1] + t).clamp(max=s["total"] - 1)
        tried = (t < rows) & (s["parents"][row] == here)
        token = s["tokens"][row].long()
        p = left[every, token]
        q = draft[every, token] if draft is not None else torch.ones_like(p)
        ok = tried & torch.where(greedy, token == best, (p > 0) & (s["uniform"][row].double() * q < p))
        rest = (left - draft).clamp(min=0) if draft is not None else left.masked_fill(one_hot(token), 0.0)
        mass = rest.sum(1, keepdim=True)
        gone = (tried & ~ok)[:, None] & (mass > 0)
        left = torch.where(ok[:, None], soft(s["logits"][row]), torch.where(gone, rest / mass, left))
        best = torch.where(ok, s["logits"][row].max(1).indices, best)
        if draft is not None:
            draft = torch.where(ok[:, None], soft(s["draft"][row]), draft)
        here = torch.where(ok, t, here)
        took.scatter_(0, row, took[row] | ok)
    s["next"].copy_(torch.where(greedy, best, (left / s["noise"].double()).argmax(1)))
    order = torch.where(took, took.cumsum(0) - 1, s["total"])
    spread = torch.full((s["total"] + 1,), -1, dtype=torch.int32, device="cuda")
    s["accepted"].copy_(spread.scatter_(0, order, torch.arange(s["total"], dtype=torch.int32, device="cuda"))[:-1])
    ends = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), took.cumsum(0)])[cu]
    s["accepted_cu"].copy_(ends)
    s["new_lens"].copy_(s["context"] + ends[1:] - ends[:-1])
    return _verify_out(s)


def _plain_weights(s):
    case = s["case"]
    hkv, group, d, page = case["hkv"], case["hq"] // case["hkv"], case["d"], case["page"]
    n, most = len(s["lens"]), max(s["rows"])
    rows = s["cu"][1:] - s["cu"][:-1]
    step = torch.arange(most, device="cuda")
    at = (s["cu"][:-1, None].long() + step[None]).clamp(max=s["total"] - 1)
    q = s["q"][at].float().reshape(n, most, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * most, d)
    k = s["k_cache"][s["tables"].long().clamp(min=0)].reshape(n, -1, hkv, d)
    slots = k.shape[1]
    scores = torch.matmul(q, k.permute(0, 2, 3, 1).float()).mul_(1.0 / math.sqrt(d)).reshape(n, hkv, group, most, slots)
    last = (s["context"] - rows)[:, None] + step[None]  # the last key that a row sees
    slot = torch.arange(slots, device="cuda")
    see = (slot[None, None] <= last[:, :, None]) & (step[None] < rows[:, None])[:, :, None]
    scores.masked_fill_(~see[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    mass = scores.sum(-1, keepdim=True)
    got = scores.div_(torch.where(mass == 0, 1.0, mass)).sum((2, 3))
    old = torch.where(slot[None] < (s["context"] - rows)[:, None], 1.0, 0.0)[:, None] * s["weights"] * case["decay"]
    s["weights"].copy_(torch.where((slot[None] < s["context"][:, None])[:, None], old + got, s["weights"]))
    return s["weights"]


def _plain_evict(s):
    case = s["case"]
    hkv, page, slots = case["hkv"], case["page"], s["weights"].shape[2]
    cuts = (s["keep"] >= 0) & (s["keep"] < s["context"])
    n = torch.where(cuts, s["keep"], s["context"])
    recent = n.clamp(max=case["recent"])
    first = torch.minimum(n - recent, torch.full_like(n, case["first"]))
    slot = torch.arange(slots, device="cuda")[None]
    inside = slot < s["context"][:, None]
    middle = (slot >= first[:, None]) & (slot < (s["context"] - recent)[:, None])
    keys = torch.where(middle[:, None], s["weights"].clamp(min=torch.finfo(torch.float32).min), -math.inf)
    order = keys.sort(dim=2, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, slot[None].expand_as(order).contiguous())
    stay = torch.where(middle[:, None], rank < (n - first - recent)[:, None, None], inside[:, None])
    place = torch.where(stay, stay.cumsum(2) - 1, slots)
    spot = torch.cat([s["kept"], s["kept"][..., :1]], 2).scatter_(2, place, slot[None].expand_as(place).to(torch.int32).contiguous())[..., :slots]
    new = slot < n[:, None]
    s["kept"].copy_(torch.where(new[:, None], spot, s["kept"]))
    source = torch.where(new[:, None], s["kept"], 0).long()
    s["weights_out"].copy_(torch.where(new[:, None], s["weights"].gather(2, source), s["weights_out"]))
    tables = s["tables"].long()
    moved = (new & cuts[:, None]).nonzero().unbind(1)  # rows that are written: sequence and slot
    from_slot = source.permute(0, 2, 1)[moved]
    head = torch.arange(hkv, device="cuda")[None]
    from_page = tables[moved[0][:, None], from_slot // page]
    to_page = tables[moved[0], moved[1] // page][:, None]
    for pool in (s["k_cache"], s["v_cache"]):
        pool[to_page, (moved[1] % page)[:, None], head] = pool[from_page, from_slot % page, head]
    s["new_lens"].copy_(torch.where(cuts, n, -1))
    return _evict_out(s)


# ---- what a pass cannot do without ----------------------------------------------------------------------------------

def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "verify":
        # behind a sequence's certain token: the target's row, the draft's, and a random number a token for the next one
        n = len(_ints(case["rows"]))
        noise = max(0, n - case["greedy"])
        return {"bytes": case["vocab"] * (n * e + (noise * e if case["draft"] else 0) + 4 * noise), "flops": 4 * case["vocab"] * n}
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "rotate":
        rows, hq = sum(_ints(case["rows"])), case["hq"]
        stored = 2 * hkv if case["store"] else 0
        return {"bytes": rows * (e * d * (2 * hq + hkv + (hkv if case["store"] else 0) + (hkv if case["k_out"] else 0) + stored) + 4 * case["rot"]),
                "flops": rows * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "weights":
        pairs = list(zip(_ints(case["rows"]), _ints(case["lens"])))
        scores = sum(t * (n - t) + t * (t + 1) // 2 for t, n in pairs)
        return {"bytes": sum(e * d * (case["hq"] * t + hkv * n) + hkv * (4 * n + (4 * (n - t) if case["decay"] else 0)) for t, n in pairs),
                "flops": 2 * d * case["hq"] * scores}
    pairs = list(zip(_ints(case["lens"]), _ints(case["keep"])))
    moved = sum(max(0, k - case["first"]) for n, k in pairs if k < n)
    return {"bytes": hkv * (sum(4 * n + 8 * min(n, k) for n, k in pairs) + 4 * e * d * moved), "flops": 0}


# ---- the definitions in 64 bits, sequence by sequence ---------------------------------------------------------------

def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = was
    return {"rotate": _exact_rotate, "verify": _exact_verify, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](case, s)


def _exact_rotate(case, s):
    half, page = case["rot"] // 2, case["page"]
    axis = [i for i, n in enumerate(_ints(case["sections"])) for _ in range(n)] if case["sections"] else [0] * half
    first = [2 * i for i in range(half)] if case["mixed"] else list(range(half))
    second = [2 * i + 1 for i in range(half)] if case["mixed"] else [half + i for i in range(half)]
    table = s["table"].double()
    out = {"q": s["q_out"].double()}
    if case["k_out"]:
        out["k"] = s["k_out"].double()
    if case["store"]:
        out.update(k_cache=s["k_cache"].double(), v_cache=s["v_cache"].double())
    at = 0
    for i, n in enumerate(s["rows"]):
        rows = slice(at, at + n)
        spot = torch.arange(s["lens"][i] - n, s["lens"][i], device="cuda")
        turned = {}
        for name, x, weight in (("q", s["q"], s["q_weight"]), ("k", s["k"], s["k_weight"])):
            x = x[rows].double()
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS) * weight.double()
            y = x.clone()
            for j in range(half):
                where = spot if s["positions"] is None else s["positions"][axis[j], rows].long()
                c, w = table[where, j][:, None], table[where, half + j][:, None]
                y[..., first[j]] = c * x[..., first[j]] - w * x[..., second[j]]
                y[..., second[j]] = w * x[..., first[j]] + c * x[..., second[j]]
            turned[name] = y
            if name in out:
                out[name][rows] = y
        if case["store"]:
            pages = s["tables"][i].long()[spot // page]
            out["k_cache"][pages, spot % page] = turned["k"]
            out["v_cache"][pages, spot % page] = s["v"][rows].double()
        at += n
    return out


def _exact_verify(case, s):
    accepted, ends, nexts, lens, at = [], [0], [], [], 0
    parents, tokens, uniform, heat = s["parents"].tolist(), s["tokens"].tolist(), s["uniform"].double().tolist(), s["temperature"].double().tolist()
    for i, n in enumerate(s["rows"]):
        here, greedy = 0, not heat[i] > 0
        path = [at]
        while True:
            target = s["logits"][at + here].double()
            best = int((target == target.max()).nonzero()[0])
            p = torch.softmax(target / (1.0 if greedy else heat[i]), 0)
            q = torch.softmax(s["draft"][at + here].double() / heat[i], 0) if s["draft"] is not None and not greedy else None
            step = None
            for t in range(here + 1, n):
                if parents[at + t] != here:
                    continue
                token = tokens[at + t]
                if greedy:
                    good = token == best
                else:
                    chance = float(p[token])
                    good = chance > 0 and uniform[at + t] * (1.0 if q is None else float(q[token])) < chance
                if good:
                    step = t
                    break
                if not greedy:
                    if q is None:
                        rest = p.clone()
                        rest[token] = 0
                    else:
                        rest = torch.clamp(p - q, min=0)
                    p = rest / rest.sum() if float(rest.sum()) > 0 else p
            if step is None:
                break
            here = step
            path.append(at + here)
        if greedy:
            nexts.append(best)
        else:
            key = p / s["noise"][i].double()
            nexts.append(int((key == key.max()).nonzero()[0]))
        accepted += path
        ends.append(len(accepted))
        lens.append(int(s["context"][i]) + len(path))
        at += n
    accepted += [-1] * (s["total"] - len(accepted))
    return {x: torch.tensor(v, dtype=torch.int32) for x, v in (("accepted", accepted), ("accepted_cu", ends), ("next", nexts), ("new_lens", lens))}


def _exact_weights(case, s):
    group, d, page, at = case["hq"] // case["hkv"], case["d"], case["page"], 0
    out = s["weights"].double()
    for i, (t, n) in enumerate(zip(s["rows"], s["lens"])):
        pages = s["tables"][i, : -(-n // page)].long()
        see = torch.arange(n, device="cuda")[None] <= torch.arange(n - t, n, device="cuda")[:, None]
        for g in range(case["hkv"]):
            k = s["k_cache"][pages, :, g].double().reshape(-1, d)[:n]
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            for h in range(g * group, (g + 1) * group):
                x = (s["q"][at:at + t, h].double() @ k.T / math.sqrt(d)).masked_fill(~see, -math.inf)
                got += torch.softmax(x, 1).sum(0)
            got[: n - t] += case["decay"] * out[i, g, : n - t]
            out[i, g, :n] = got
        at += t
    return out


def _exact_evict(case, s):
    page, lens, keep = case["page"], s["lens"], s["keep"].tolist()
    k, v, kept, weights_out = s["k_cache"].double(), s["v_cache"].double(), s["kept"].clone(), s["weights_out"].double()
    new_lens, weights, tables = [], s["weights"].double().cpu(), s["tables"].long()
    for i, n in enumerate(lens):
        cut = 0 <= keep[i] < n
        m = keep[i] if cut else n
        new_lens.append(m if cut else -1)
        recent = min(case["recent"], m)
        first = min(case["first"], m - recent)
        for g in range(case["hkv"]):
            w = weights[i, g].tolist()
            top = sorted(range(first, n - recent), key=lambda j: (-w[j], j))[: m - first - recent]
            stay = torch.tensor(list(range(first)) + sorted(top) + list(range(n - recent, n)), dtype=torch.long, device="cuda")
            kept[i, g, :m] = stay.to(torch.int32)
            weights_out[i, g, :m] = weights[i, g].to(weights_out.device)[stay]
            if cut:
                to = torch.arange(m, device="cuda")
                for pool in (k, v):
                    pool[tables[i, to // page], to % page, g] = pool[tables[i, stay // page], stay % page, g]
    return {"k_cache": k, "v_cache": v, "weights_out": weights_out, "kept": kept, "new_lens": torch.tensor(new_lens, dtype=torch.int32)}
