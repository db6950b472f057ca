"""The Python entry points refuse a table whose rows are not as wide as the
parameters say: read as another width, its rows would be other rows' entries."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import build, ops


class Passed(Exception):
    """Every check of the arguments passed."""


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    """Tensors of the CPU (device -1) go through the checks; nothing is called."""
    build.build()
    ops.load()

    def call(name, dev, stream, *args):
        raise Passed(name)
    monkeypatch.setattr(ops, "_call", call)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


P = dict(num_seqs=3, num_q_heads=4, num_kv_heads=2, head_dim=64, page_size=16, num_pages=6, max_blocks_per_seq=4,
         max_context_len=64, dtype="bf16", out_dtype="bf16")


def calls(table=None, mask=None, pairs=None):
    """Each entry point with the given table, mask and pairs, the others right."""
    p, r = ops.make_params(**P), ops.make_rows(5, 3)
    q, k, pool = (torch.zeros(*s, 64, dtype=torch.bfloat16) for s in ((5, 4), (5, 2), (6, 16, 2)))
    t, m, w = i32(3, 4) if table is None else table, i32(5, 1) if mask is None else mask, i32(3, 2) if pairs is None else pairs
    ws, ref, lens = torch.zeros(1, dtype=torch.uint8), i32(6), i32(3)
    return {"tree": lambda: ops.tree(p, r, q, k, k, i32(4), m, pool, pool, t, lens, out=q.clone(), workspace=ws),
            "store": lambda: ops.store(p, r, k, k, i32(4), pool, pool, t, lens),
            "resize": lambda: ops.pages_resize(p, ref, t, lens, lens, w, ws),
            "fork": lambda: ops.pages_fork(p, ref, t, lens, i32(1), i32(1)),
            "compact": lambda: ops.pages_compact(p, ref, t, lens, w, i32(1), ws),
            "copy": lambda: ops.pages_copy(p, pool, pool, w)}


def test_tables_of_the_right_width_pass():
    for kw in (dict(), dict(table=i32(12)), dict(table=i32(7, 4)), dict(mask=i32(9)), dict(mask=i32(8, 1)), dict(pairs=i32(6)),
               dict(pairs=i32(5, 2))):
        for call in calls(**kw).values():
            with pytest.raises(Passed):
                call()


@pytest.mark.parametrize("kw,names", [(dict(table=i32(3, 8)), ("tree", "store", "resize", "fork", "compact")),
                                      (dict(table=i32(6, 2)), ("tree", "store", "resize", "fork", "compact")),
                                      (dict(mask=i32(5, 2)), ("tree",)), (dict(pairs=i32(2, 3)), ("resize", "compact", "copy")),
                                      (dict(pairs=i32(2, 4)), ("resize", "compact", "copy"))])
def test_tables_of_another_width_are_refused(kw, names):
    for name, call in calls(**kw).items():
        with pytest.raises(ValueError if name in names else Passed):
            call()
