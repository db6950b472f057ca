"""Prompt and tree attention where one key outweighs each other by far and they,
many of them, still count together: a weight is rounded relative to the row's
largest, not to nothing.

Each key of weight w adds, to what serving_ref.bound counts, what an fp16 weight
may lose to the type's least subnormal: half of its step, 2^-25, where the row's
largest weight is 2^10 at least, so 2^-35 of the largest for each key."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gqa_02_gb300 import build, ops
import serving_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]
SCALE = 0.125


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.load()


def keys(n, gap, top, d, dtype):
    """Key `top` scores 0 and every other one 2^-gap of its weight (q is 1 in dim 0)."""
    k = torch.zeros(n, 1, d, dtype=torch.float64)
    k[:, 0, 0] = -gap * math.log(2.0) / SCALE
    k[top, 0, 0] = 0.0
    return k.to(ref.DT[dtype]).cuda()


def check(out, q, k, v, see, out_dtype, dtype, what):
    n = k.shape[0]
    want, weight = ref.attend(q.double(), k.double(), v.double(), see, SCALE)
    tol = ref.bound(want, weight, q.double()[:1], k.double(), SCALE, n, dtype, out_dtype)
    if dtype == "f16":
        tol = tol + n * 2.0 ** -35 * float(v.abs().max())
    assert float((want.abs() / tol).median()) > 20, "the bound would pass zeros"
    ref.assert_close(out, want, tol, what)


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("gap", (20.0, 25.5, 29.0))
@pytest.mark.parametrize("top", ("first", "middle", "draft"))
def test_tree_of_a_long_history(dtype, out_dtype, gap, top):
    n, m, hq, d, page = 1 << 17, 3, 4, 64, 32
    gen = torch.Generator().manual_seed(21)
    pool = ref.Pool([n], page, 1, d, dtype, gen)
    every = keys(n + m, gap, {"first": 0, "middle": n // 2 + 5, "draft": n}[top], d, dtype)
    values = (1.0 + torch.rand(n + m, 1, d, generator=gen)).to(ref.DT[dtype]).cuda()
    values[{"first": 0, "middle": n // 2 + 5, "draft": n}[top]] = 0.0
    order = pool.tables[0, :n // page].long()
    for x, y in zip(pool.kv, (every, values)):
        x[order] = y[:n].reshape(-1, page, 1, d)
    q = torch.zeros(m, hq, d, dtype=ref.DT[dtype], device="cuda")
    q[:, :, 0] = 1.0
    mask = torch.tensor([[1], [3], [7]], dtype=torch.int32, device="cuda")
    p = pool.params(hq, out_dtype=out_dtype, scale=SCALE)
    out = ops.tree(p, ops.make_rows(m, m), q, every[n:].contiguous(), values[n:].contiguous(), ref.cu([m]), mask, pool.k, pool.v,
                   pool.tables, pool.context)
    see = torch.cat([torch.ones(m, n, dtype=torch.bool, device="cuda"), ref.bits(mask, 0, m)], 1)
    for h in range(hq):
        check(out[:, h], q[:, h], every[:, 0], values[:, 0], see, out_dtype, dtype, f"2^-{gap} head {h}")


@pytest.mark.parametrize("dtype,out_dtype", TYPES[1:])
@pytest.mark.parametrize("gap", (20.0, 25.5))
@pytest.mark.parametrize("top", (0, 20001))
def test_long_prompt(dtype, out_dtype, gap, top):
    n, d = 40000, 64
    gen = torch.Generator().manual_seed(22)
    k = keys(n, gap, top, d, dtype)
    v = (1.0 + torch.rand(n, 1, d, generator=gen)).to(ref.DT[dtype]).cuda()
    v[top] = 0.0
    q = torch.zeros(n, 1, d, dtype=ref.DT[dtype], device="cuda")
    q[:, :, 0] = 1.0
    p = ops.prompt_params(num_seqs=1, num_q_heads=1, num_kv_heads=1, head_dim=d, scale=SCALE, dtype=dtype, out_dtype=out_dtype)
    out = ops.prompt(p, ops.make_rows(n, n), q, k, v, ref.cu([n]))
    rows = slice(n - 40, n)
    see = torch.arange(n, device="cuda")[None] <= torch.arange(n - 40, n, device="cuda")[:, None]
    check(out[rows, 0], q[rows, 0], k[:, 0], v[:, 0], see, out_dtype, dtype, f"2^-{gap}")
