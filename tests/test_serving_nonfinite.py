"""Prompt and tree attention beside one value in V that is not finite: an element
of the output depends on the weights, which V has no part in, and on its own dim
of V, so every other dim, row and head keeps its bits.  The shapes give a CTA
one unit after another, most of one row tile and several key tiles, so that a
row that takes long to put right is followed by another unit's products."""
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
VALUES = (float("nan"), float("inf"), -float("inf"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.load()


def normal(gen, *shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(ref.DT[dtype])


def check(out, clean, sees, dim, value):
    """`sees` [rows][heads]: which rows attend the value that stands in dim `dim`."""
    seen = out[sees][:, dim]
    assert (seen.isnan() if math.isnan(value) else seen == value).all()
    want = clean.clone()
    want[..., dim] = torch.where(sees, out[..., dim], clean[..., dim])
    same = (out == want) | (out.isnan() & want.isnan())
    assert same.all(), f"{int((~same).sum())} other elements"


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("d,dims", [(64, (3, 40)), (128, (5, 40, 70, 100))])
def test_prompt_keeps_the_other_dims(dtype, out_dtype, d, dims):
    lens, hq, hkv = [2300, 200], 16, 2
    gen = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = normal(gen, 2500, hq, d, dtype=dtype), normal(gen, 2500, hkv, d, dtype=dtype), normal(gen, 2500, hkv, d, dtype=dtype)
    p = ops.prompt_params(num_seqs=2, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=dtype, out_dtype=out_dtype)
    r, c = ops.make_rows(2500, 2300), ref.cu(lens)
    clean = ops.prompt(p, r, q, k, v, c)
    want, tol = ref.prompt_ref(q[2300:], k[2300:], v[2300:], [200], p.scale, dtype, out_dtype)
    ref.assert_close(clean[2300:], want, tol)
    for i, dim in enumerate(dims):
        for j, value in ((0, VALUES[i % 3]), (1500, float("nan"))):
            g, kept = i % 2, v[j, i % 2, dim].clone()
            v[j, g, dim] = value
            sees = torch.zeros(2500, hq, dtype=torch.bool, device="cuda")
            sees[j:2300, g * 8:(g + 1) * 8] = True
            for _ in range(3):
                check(ops.prompt(p, r, q, k, v, c), clean, sees, dim, value)
            v[j, g, dim] = kept


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("d,dims", [(64, (3, 40)), (128, (5, 40, 70, 100))])
def test_tree_keeps_the_other_dims(dtype, out_dtype, d, dims):
    """The value stands in a page of the history, or among the drafts."""
    n, hq, hkv, page = 24, 32, 8, 16
    lens, drafts = [300 + (i * 97) % 900 for i in range(n)], [4 + i % 13 for i in range(n)]
    gen = torch.Generator().manual_seed(d)
    pool = ref.Pool(lens, page, hkv, d, dtype, gen)
    total = sum(drafts)
    dev = torch.Generator(device="cuda").manual_seed(d + 1)
    q, k, v = normal(dev, total, hq, d, dtype=dtype), normal(dev, total, hkv, d, dtype=dtype), normal(dev, total, hkv, d, dtype=dtype)
    mask = ref.random_mask(drafts, 1, gen)
    p, r, c = pool.params(hq, out_dtype=out_dtype), ops.make_rows(total, max(drafts)), ref.cu(drafts)
    ws = torch.empty(ops.tree_workspace_size(p, r), dtype=torch.uint8, device="cuda")

    def go():
        return ops.tree(p, r, q, k, v, c, mask, pool.k, pool.v, pool.tables, pool.context, workspace=ws)
    clean = go()
    want, tol = ref.tree_ref(q, k, v, drafts, mask, *pool.kv, pool.tables, lens, p.scale, dtype, out_dtype)
    ref.assert_close(clean, want, tol)
    for i, dim in enumerate(dims):
        value = VALUES[i % 3]
        for s in (0, 11):
            g, at, m = (3 * i + s) % hkv, sum(drafts[:s]), drafts[s]
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            for place in (2, lens[s] - 1, "draft"):
                sees = torch.zeros(total, hq, dtype=torch.bool, device="cuda")
                if place == "draft":
                    spot = v[at + 1, g]
                    sees[at:at + m, heads] = ref.bits(mask, at, m)[:, 1:2]
                else:
                    spot = pool.kv[1][int(pool.tables[s, place // page]), place % page, g]
                    sees[at:at + m, heads] = True
                kept = spot[dim].clone()
                spot[dim] = value
                check(go(), clean, sees, dim, value)
                spot[dim] = kept


@pytest.mark.parametrize("dtype,out_dtype", TYPES[1:])
def test_infinities_everywhere(dtype, out_dtype):
    """Every row sums what it sees: an infinity of its sign, or NaN where it sees both, in every dim."""
    n, hq, hkv, d = 3000, 4, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = normal(gen, n, hq, d, dtype=dtype), normal(gen, n, hkv, d, dtype=dtype), normal(gen, n, hkv, d, dtype=dtype)
    p = ops.prompt_params(num_seqs=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=dtype, out_dtype=out_dtype)
    first = torch.randint(0, n, (hkv, d), generator=gen, device="cuda")   # from here on +inf
    other = torch.randint(0, 4 * n, (hkv, d), generator=gen, device="cuda")  # here -inf
    at = torch.arange(n, device="cuda")[:, None, None]
    clean = ops.prompt(p, ops.make_rows(n, n), q, k, v, ref.cu([n]))
    v = torch.where(at >= first, torch.full_like(v, float("inf")), v)
    v = torch.where(at == other, torch.full_like(v, -float("inf")), v)
    out = ops.prompt(p, ops.make_rows(n, n), q, k, v, ref.cu([n]))
    up, down = ((v == x).cumsum(0) > 0 for x in (float("inf"), -float("inf")))
    up, down = (x.repeat_interleave(hq // hkv, 1) for x in (up, down))
    want = torch.where(up, torch.full_like(clean, float("inf")), clean)
    want = torch.where(down, torch.full_like(clean, -float("inf")), want)
    want = torch.where(up & down, torch.full_like(clean, float("nan")), want)
    same = (out == want) | (out.isnan() & want.isnan())
    assert same.all(), f"{int((~same).sum())} elements"
