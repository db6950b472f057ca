"""An exchange of pa_verify that is given up: the status says so, every CTA of the cluster ends, and the next call is right.

The wait that runs out is made on the host's word (debug_timeout): the first CTA of each sequence's cluster gives up at
once on its first exchange, the others go on to the next one and send to it while it leaves."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import cu
from test_step_verify import check, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab,draft,chain", [
    ((3,), 300, True, True),            # one CTA
    ((4,), 9000, False, True),          # a cluster of four
    ((6,), 131072, True, False),        # of sixteen
    ((5,) * 40, 20000, True, True),     # more sequences than widest clusters
    ((1, 0, 7), 50021, False, False)])  # no children; no rows
def test_a_wait_that_runs_out_leaves_the_context_usable(rows, vocab, draft, chain):
    x = problem(rows, vocab, "bf16", draft, chain, 71)
    p, r = ops.verify_params(num_seqs=len(rows), dtype="bf16"), ops.make_rows(sum(rows), max(rows))
    p.debug_timeout = 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, ends, _, _ = ops.verify(p, r, x["logits"], x["draft"], x["tokens"], x["parents"], cu(x["rows"]), x["heat"], x["uniform"], x["noise"],
                               dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == ops.PA_DEV_TIMEOUT
    ends = ends.tolist()
    assert all(0 <= b - a <= n for a, b, n in zip(ends, ends[1:], rows))  # void, but counts still
    check(x, near=1)
