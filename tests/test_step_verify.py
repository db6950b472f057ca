"""pa_verify against a walk of the definition in 64 bits."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import DT, cu

pytestmark = pytest.mark.gpu


def walk(logits, draft, tokens, parents, heat, uniform, noise):
    """(accepted rows, next token, margin) of one sequence: how near, relatively,
    a comparison of computed numbers came to going the other way."""
    greedy, here, path, margin, n = not heat > 0, 0, [0], math.inf, len(tokens)
    while True:
        row = logits[here].double()
        top = row.max()
        if not bool((row <= torch.finfo(torch.float32).max).all()) or not bool(top > -math.inf):
            return path, -1, margin
        p = torch.softmax(row / (1.0 if greedy else heat), 0)
        children = [t for t in range(here + 1, n) if parents[t] == here and 0 <= tokens[t] < len(row)]
        q = None
        if draft is not None and not greedy and children:
            other = draft[here].double()
            if not bool((other <= torch.finfo(torch.float32).max).all()) or not bool(other.max() > -math.inf):
                return path, -1, margin
            q = torch.softmax(other / heat, 0)
        best, step = int((row == top).nonzero()[0]), None
        for t in children:
            c = tokens[t]
            if greedy:
                good = c == best
            else:
                a, b = float(uniform[t]) * (1.0 if q is None else float(q[c])), float(p[c])
                good = b > 0 and a < b
                if a or b:
                    margin = min(margin, abs(a - b) / max(a, b))
            if good:
                step = t
                break
            if not greedy:
                rest = p.clone()
                if q is None:
                    rest[c] = 0
                else:
                    rest = torch.clamp(p - q, min=0)
                p = rest / rest.sum() if float(rest.sum()) > 0 else p
        if step is None:
            break
        here = step
        path.append(here)
    if greedy:
        return path, best, margin
    key = p / noise.double()
    two = key.topk(min(2, len(key))).values
    if len(two) == 2:
        margin = min(margin, float((two[0] - two[1]) / two[0]))
    return path, int((key == two[0]).nonzero()[0]), margin


def problem(rows, vocab, dtype, draft, chain, seed, spread=3.0, stride=0):
    gen = torch.Generator().manual_seed(seed)
    total, dt, wide = sum(rows), DT[dtype], stride or vocab
    target = spread * torch.randn(total, wide, generator=gen)
    other = (target + 0.5 * torch.randn(total, wide, generator=gen)).to(dt).cuda()[:, :vocab]
    parents, at = [], 0
    for n in rows:
        parents += [t - 1 if chain else (int(torch.randint(0, t, (1,), generator=gen)) if t else 0) for t in range(n)]
        at += n
    starts = [sum(rows[:i]) for i in range(len(rows))]
    seq = [i for i, n in enumerate(rows) for _ in range(n)]
    tokens = []
    for i in range(total):
        row = other[starts[seq[i]] + max(parents[i], 0)].double().cpu()
        tokens.append(int(torch.multinomial(torch.softmax(row, 0), 1, generator=gen)))
    return dict(rows=rows, logits=target.to(dt).cuda()[:, :vocab], draft=other if draft else None, tokens=torch.tensor(tokens, dtype=torch.int32).cuda(),
                parents=torch.tensor(parents, dtype=torch.int32).cuda(), heat=(0.6 + torch.rand(len(rows), generator=gen)).cuda(),
                uniform=torch.rand(total, generator=gen).cuda(),
                noise=torch.empty(len(rows), vocab).exponential_(generator=gen).clamp_(min=1e-7).cuda(), stride=stride)


def call(x, context=None, status=None, **kw):
    p = ops.verify_params(num_seqs=len(x["rows"]), dtype={v: k for k, v in DT.items()}[x["logits"].dtype])
    r = ops.make_rows(x["logits"].shape[0], max(max(x["rows"]), 1), q_stride=x["stride"], k_stride=x["stride"])
    return ops.verify(p, r, x["logits"], x["draft"], x["tokens"], x["parents"], cu(x["rows"]), x["heat"], x["uniform"], x["noise"],
                      context_lens=context, dev_status=status, **kw)


def check(x, near=0):
    """Compares a call with the walk; `near` sequences at most may be too near a border to tell."""
    context = torch.arange(7, 7 + len(x["rows"]), dtype=torch.int32, device="cuda")
    accepted, ends, nexts, lens = (t.tolist() for t in call(x, context))
    at, close, want_ends = 0, 0, [0]
    for s, n in enumerate(x["rows"]):
        mine = slice(at, at + n)
        got = (accepted[ends[s]:ends[s + 1]], nexts[s])
        if n == 0:
            assert got == ([], -1)
        else:
            path, token, margin = walk(x["logits"][mine], None if x["draft"] is None else x["draft"][mine], x["tokens"][mine].tolist(),
                                       x["parents"][mine].tolist(), float(x["heat"][s]), x["uniform"][mine], x["noise"][s])
            # sums of fp32 terms, each within 2^-20 of its value: what is further apart cannot be confused
            if margin < 2.0 ** -16:
                close += 1
            else:
                assert got == ([at + t for t in path], token), (s, got, path, token, margin)
        at += n
        want_ends.append(ends[s] + len(got[0]))
        assert lens[s] == 7 + s + len(got[0])
    assert ends == want_ends and all(a == -1 for a in accepted[ends[-1]:]) and close <= near
    return accepted, ends, nexts


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab,draft,chain", [
    ((1,), 1, False, True), ((1, 1), 2, True, True), ((2, 0, 5), 7, True, True), ((5, 5, 1), 1000, False, True), ((6, 3, 9, 1), 4099, True, True),
    ((20, 1, 33, 64), 515, True, False), ((64, 7), 2048, False, False), ((3,) * 40, 999, True, False), ((200, 1024), 130, True, False), ((9,), 70001, True, False)])
def test_walks(rows, vocab, draft, chain, dtype):
    for seed in range(3):
        check(problem(rows, vocab, dtype, draft, chain, seed), near=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_rows_and_odd_bases(dtype):
    x = problem((4, 6, 2), 1001, dtype, True, False, 9, stride=1003)
    check(x)
    for k in ("logits", "draft"):  # a base that no 16-byte boundary holds
        flat = torch.zeros(x[k].shape[0] * 1003 + 1, dtype=x[k].dtype, device="cuda")
        flat[1:].view(-1, 1003)[:, :1001] = x[k]
        x[k] = flat[1:].view(-1, 1003)[:, :1001]
    check(x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["logits", "draft", "noise"])
@pytest.mark.parametrize("vocab", [1000, 40003])
def test_each_base_on_its_own_boundary(which, vocab, dtype):
    x = problem((4, 6, 2), vocab, dtype, True, False, 19)
    flat = torch.zeros(x[which].numel() + 1, dtype=x[which].dtype, device="cuda")
    flat[1:] = x[which].reshape(-1)
    x[which] = flat[1:].view(x[which].shape)
    check(x)


@pytest.mark.parametrize("seqs", [8, 9, 17, 26, 40, 80])
def test_as_many_sequences_as_the_gpu_holds_and_more(seqs):
    check(problem((2,) * seqs, 24600, "bf16", True, True, 60 + seqs), near=1)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 300007), ("f32", 150001), ("f16", 8)])
def test_vocabularies_beyond_the_slots(dtype, vocab):
    check(problem((3, 1, 5), vocab, dtype, True, False, 21), near=1)
    check(problem((2,) * 160, vocab // 40 + 1, dtype, True, True, 22), near=2)  # one CTA a sequence


def test_captured_and_replayed():
    """A captured call takes the rows, lengths and numbers that it finds; two graphs replayed in turn do not disturb one another."""
    graphs = []
    for seed in (30, 31):
        x = problem((5, 9, 1, 30), 5003, "bf16", True, False, seed)
        rows = cu(x["rows"])
        p, r = ops.verify_params(num_seqs=4, dtype="bf16"), ops.make_rows(x["logits"].shape[0], 30)
        out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (x["logits"].shape[0], 5, 4)]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                ops.verify(p, r, x["logits"], x["draft"], x["tokens"], x["parents"], rows, x["heat"], x["uniform"], x["noise"],
                           accepted=out[0], accepted_cu=out[1], next_tokens=out[2])
        graphs.append((graph, x, rows, out))
    torch.cuda.synchronize()
    for counts in ((5, 9, 1, 30), (1, 0, 4, 2)):
        for graph, x, rows, out in graphs:
            rows.copy_(cu(counts))
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        for graph, x, rows, out in graphs:
            ends, at = out[1].tolist(), 0
            for s, n in enumerate(counts):
                mine = slice(at, at + n)
                if n:
                    parents = [p if 0 <= p < t else -1 for t, p in enumerate(x["parents"][mine].tolist())]
                    path, token, margin = walk(x["logits"][mine], x["draft"][mine], x["tokens"][mine].tolist(), parents, float(x["heat"][s]),
                                               x["uniform"][mine], x["noise"][s])
                    if margin > 2.0 ** -16:
                        assert out[0][ends[s]:ends[s + 1]].tolist() == [at + t for t in path] and int(out[2][s]) == token
                else:
                    assert ends[s] == ends[s + 1] and int(out[2][s]) == -1
                at += n


def test_hot_and_cold_temperatures():
    x = problem((4, 4, 4), 700, "f32", True, True, 23)
    x["heat"][0], x["heat"][1], x["heat"][2] = 1e-30, 1e30, 50.0
    check(x, near=1)
    x["logits"][:] = -3.4028234e38  # masked everywhere: uniform
    x["heat"][:] = 1.0
    check(x, near=1)


def test_an_infinite_temperature_makes_finite_logits_alike():
    x = problem((4, 4), 700, "f32", True, True, 24)
    x["logits"][:, ::3] = -math.inf
    x["draft"][:, ::3] = -math.inf
    x["tokens"][:] = 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for heat in (math.inf, 3.4028234e38):
        x["heat"][:] = heat
        accepted, ends, nexts, _ = call(x, status=status)
        assert int(status) == 0 and ends.tolist() == [0, 4, 8]  # p = q
        for s, token in enumerate(nexts.tolist()):  # the smallest noise of a token that is not masked
            masked = x["noise"][s].clone()
            masked[::3] = math.inf
            assert token == int(masked.argmin())


def test_greedy_and_ties():
    x = problem((6, 9, 30), 333, "bf16", True, False, 3)
    x["heat"][0], x["heat"][1] = 0.0, -1.0
    x["logits"][:, 200] = x["logits"][:, 100] = 90.0  # the lower of two equal ones wins
    x["draft"][:6] = float("nan")  # not read
    x["uniform"][:6] = float("nan")
    x["noise"][:2] = float("nan")
    x["tokens"][0:6] = 100
    x["tokens"][6:15] = 200
    accepted, ends, nexts = check(x)
    assert ends[1] >= 2 and nexts[0] == 100 and ends[2] - ends[1] == 1 and nexts[1] == 100


def test_same_distribution_accepts_all_and_repeats():
    x = problem((8, 8), 500, "f32", True, True, 4)
    x["draft"] = x["logits"].clone()
    accepted, ends, _ = check(x)
    assert ends == [0, 8, 16] and accepted == list(range(16))
    # the same token twice under one parent, rejected both times
    for draft in (True, False):
        x = problem((5,), 64, "f32", draft, False, 5)
        x["parents"][:] = 0
        x["tokens"][1:] = 3
        x["logits"][:, 3] = -2.0
        if draft:
            x["draft"][:, 3] = 9.0
        x["uniform"][:] = 0.999
        accepted, ends, nexts = check(x)
        assert ends == [0, 1] and nexts[0] != 3


def test_infinite_logits_are_probabilities_of_zero():
    x = problem((4, 4, 4), 300, "f16", True, True, 6)
    x["logits"][:, ::2] = -math.inf
    x["draft"][:, 1::7] = -math.inf
    x["uniform"][4:8] = 0.0
    check(x)
    x["logits"][:, :] = -math.inf
    x["logits"][:, 17] = 1.0
    _, _, nexts = check(x)
    assert nexts == [17, 17, 17]


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_rows_without_a_distribution_end_the_walk(value):
    x = problem((3, 3, 3), 257, "bf16", True, True, 7)
    x["draft"] = x["logits"].clone()  # all accepted otherwise
    x["logits"][0, 256] = value
    x["draft"][4, 0] = value
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    accepted, ends, nexts, lens = call(x, status=status)
    assert int(status) == ops.PA_DEV_BAD_VALUE and lens is None
    assert ends.tolist() == [0, 1, 3, 6] and accepted.tolist() == [0, 3, 4, 6, 7, 8, -1, -1, -1] and nexts.tolist()[:2] == [-1, -1]
    x["logits"][:] = -math.inf
    status.zero_()
    _, ends, nexts, _ = call(x, status=status)
    assert int(status) == ops.PA_DEV_BAD_VALUE and nexts.tolist() == [-1] * 3 and ends.tolist() == [0, 1, 2, 3]


def test_bad_drafts_are_passed_over():
    x = problem((6, 6), 100, "f32", False, False, 8)
    x["parents"][:] = 0
    x["uniform"][:] = 0.0
    x["tokens"][1], x["tokens"][2], x["parents"][3] = -1, 100, 3  # tokens outside, its own parent
    x["parents"][7], x["parents"][8] = 5, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    accepted, ends, _, _ = call(x, status=status)
    assert int(status) == ops.PA_DEV_BAD_INDEX and accepted.tolist()[:4] == [0, 4, 6, 9] and ends.tolist() == [0, 2, 4]


def test_noise_that_chooses_nothing():
    x = problem((1, 1), 50, "f32", False, True, 9)
    x["noise"][0] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, _, nexts, _ = call(x, status=status)
    assert int(status) == ops.PA_DEV_BAD_VALUE and nexts[0] == -1 and nexts[1] >= 0


def test_rows_out_of_range():
    x = problem((3, 3, 3), 50, "f32", False, True, 10)
    p, r = ops.verify_params(num_seqs=3, dtype="f32"), ops.make_rows(9, 3)
    for starts, counts in (([0, 3, 2, 5], [True, False, True]), ([0, 3, 7, 9], [True, False, True]), ([0, 3, 6, 10], [True, True, False])):
        # a sequence that begins inside a chain has rows whose parents are none of its own
        bad = any(not 0 <= int(x["parents"][a + t]) < t for ok, a, b in zip(counts, starts, starts[1:]) for t in range(1, b - a if ok else 0))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        _, ends, nexts, _ = ops.verify(p, r, x["logits"], None, x["tokens"], x["parents"], torch.tensor(starts, dtype=torch.int32, device="cuda"),
                                       x["heat"], x["uniform"], x["noise"], dev_status=status)
        assert int(status) == ops.PA_DEV_BAD_LEN | (ops.PA_DEV_BAD_INDEX if bad else 0)
        assert [b > a for a, b in zip(ends.tolist(), ends.tolist()[1:])] == counts and [t >= 0 for t in nexts.tolist()] == counts


def test_no_rows_at_all():
    x = problem((1,), 50, "f32", False, True, 10)
    p, r = ops.verify_params(num_seqs=2, dtype="f32"), ops.make_rows(0, 0)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    _, ends, nexts, lens = ops.verify(p, r, x["logits"][:0], None, none, none, cu([0, 0]), torch.ones(2, device="cuda"), x["uniform"][:0],
                                      torch.ones(2, 50, device="cuda"), context_lens=torch.tensor([4, 5], dtype=torch.int32, device="cuda"))
    assert ends.tolist() == [0, 0, 0] and nexts.tolist() == [-1, -1] and lens.tolist() == [4, 5]


def test_no_rows_need_no_pointers_of_rows():
    p, r, b = ops.verify_params(num_seqs=2, dtype="bf16"), ops.make_rows(0, 0), 2
    ends, nexts, status = (torch.full((n,), 9, dtype=torch.int32, device="cuda") for n in (b + 1, b, 1))
    status.zero_()
    starts = cu([0, 0])
    assert ops.load().pa_verify(p, r, 50, None, None, None, None, starts.data_ptr(), None, None, None, None, None, ends.data_ptr(),
                                nexts.data_ptr(), None, status.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert ends.tolist() == [0, 0, 0] and nexts.tolist() == [-1, -1] and int(status) == 0


def test_many_sequences_join_in_order():
    rows = [(i * 7) % 4 for i in range(1500)]
    check(problem(rows, 40, "f32", True, True, 11), near=3)


def test_first_tokens_follow_the_target():
    """One draft from q, then the token behind it where it was rejected: together they are a draw from p.  With n
    draws a frequency has a deviation of sqrt(p (1 - p) / n) at most; six of them are passed by one in 10^8."""
    vocab, n = 6, 4000
    gen = torch.Generator().manual_seed(12)
    p, q = (torch.softmax(torch.randn(vocab, generator=gen), 0) for _ in range(2))
    x = problem((2,) * n, vocab, "f32", True, True, 13)
    x["logits"][:], x["draft"][:], x["heat"][:] = p.log().cuda(), q.log().cuda(), 1.0
    x["tokens"][1::2] = torch.multinomial(q, n, replacement=True, generator=gen).to(torch.int32).cuda()
    _, ends, nexts, _ = call(x)
    took = (ends[1:] - ends[:-1]) == 2
    first = torch.where(took, x["tokens"][1::2], nexts).cpu()
    share = torch.bincount(first.long(), minlength=vocab) / n
    assert bool(((share - p).abs() <= 6 * (p * (1 - p) / n).sqrt()).all())
