"""pa_verify where little or nothing is left of the target's distribution after a rejection."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from test_step_verify import call, check, problem

pytestmark = pytest.mark.gpu
N = 64  # sequences: the rounding of some sums' reciprocals shows in one of six


def family(children, vocab, dtype, seed):
    """N sequences, each a token with `children` drafts under it."""
    x = problem((1 + children,) * N, vocab, dtype, True, False, seed)
    x["parents"][:] = 0
    x["uniform"][:] = 0.5
    return x, x["tokens"].view(N, 1 + children), x["logits"].view(N, 1 + children, vocab), x["draft"].view(N, 1 + children, vocab)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [500, 20011])
@pytest.mark.parametrize("masked", [1, 2])
def test_nothing_is_left_where_both_distributions_are_alike(masked, vocab, dtype):
    """A draft that the target and the draft rule out is rejected; p - q is 0 everywhere, so p stays as it is and
    the next sibling is taken by it."""
    x, tokens, logits, draft = family(masked + 1, vocab, dtype, 81)
    logits[:, :, :masked] = -math.inf
    draft.copy_(logits)
    for i in range(masked):
        tokens[:, 1 + i] = i
    tokens[:, -1] = logits[:, 0].argmax(1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    accepted, ends, _, _ = call(x, status=status)
    assert int(status) == 0
    assert ends.tolist() == list(range(0, 2 * N + 1, 2))
    assert accepted[:2 * N].view(N, 2)[:, 1].tolist() == [(masked + 2) * (s + 1) - 1 for s in range(N)]
    check(x, near=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_next_token_where_nothing_is_left(dtype):
    """All drafts ruled out by both: the next token comes from p."""
    x, tokens, logits, draft = family(3, 3001, dtype, 82)
    logits[:, :, :3] = -math.inf
    draft.copy_(logits)
    tokens[:, 1:] = torch.arange(3, device="cuda", dtype=torch.int32)
    accepted, ends, nexts = check(x, near=1)
    assert ends == list(range(N + 1)) and min(nexts) >= 3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_token_is_left(dtype):
    """The two differ in one token, which the target likes better: it is all that is left of p."""
    x, tokens, logits, draft = family(3, 1000, dtype, 83)
    logits[:, :, 0] = -math.inf
    draft.copy_(logits)
    logits[:, :, 1] = 6.0
    draft[:, :, 1] = 2.0
    tokens[:, 1:] = torch.tensor([0, 5, 1], device="cuda", dtype=torch.int32)  # ruled out, another, the one
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    accepted, ends, _, _ = call(x, status=status)
    assert int(status) == 0 and ends.tolist() == list(range(0, 2 * N + 1, 2))
    assert accepted[:2 * N].view(N, 2)[:, 1].tolist() == [4 * s + 3 for s in range(N)]
    tokens[:, 3] = 7  # nor is this: the next token is the one
    accepted, ends, nexts, _ = call(x, status=status)
    assert ends.tolist() == list(range(N + 1)) and nexts.tolist() == [1] * N and int(status) == 0
