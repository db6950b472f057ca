"""pa_key_weights of scores of any finite size, and of keys that hold their type's lowest value.

Scores are whole numbers times a power of two, so that what is off is the softmax.  u = 2^-24, half a step of fp32.
Scores far apart (more than 150 in base 2) weigh 1 / (the number of the largest ones) or nothing: only the sums of ones
below and of C columns above are off, (n + C) u, and the reciprocal, the product and 2^0, 8 u.  Nearer ones have
exponents that are off by (9 X + 50) u, X the largest score in base 2, and so their weights by 0.7 of that, relatively,
and rescaled sums, 6 u for each of 20 joins and a tile of 16 keys."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import DT, Pool, assert_close, cu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ROWS = [((1, 1, 1), (200, 33, 64), 4, 2), ((3, 1), (150, 64), 6, 1), ((40, 17), (300, 64), 6, 2), ((200,), (200,), 3, 3)]


def compare(q, k, pool, rows, scale, bound, dtype):
    """q, k in 64 bits; bound(scores in base 2 of a head, seen, keys, columns) -> relative bound of its weights."""
    hq, hkv = q.shape[1], k.shape[2]
    group = hq // hkv
    weights = torch.full((len(rows), hkv, pool.blocks * pool.page), math.nan, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p, r = pool.params(hq, scale=scale), ops.make_rows(sum(rows), max(rows))
    ops.key_weights(p, r, q.to(DT[dtype]).contiguous(), cu(rows), pool.k, pool.tables, pool.context, weights, decay=0.0, dev_status=status)
    assert int(status) == 0
    at = 0
    for s, (n, L) in enumerate(zip(rows, pool.lens)):
        spot = torch.arange(L, device="cuda")
        kk = k[pool.tables[s].long()[spot // pool.page], spot % pool.page]
        see = spot[None] <= torch.arange(L - n, L, device="cuda")[:, None]
        for g in range(hkv):
            x = torch.einsum("thd,jd->htj", q[at:at + n, g * group:(g + 1) * group], kk[:, g]) * scale
            w = torch.softmax(x.masked_fill(~see, -math.inf), 2)
            rel = bound(x * math.log2(math.e), see, L, n * group)
            assert_close(weights[s, g, :L], w.sum((0, 1)), (rel * w).sum((0, 1)) + 1e-30, f"sequence {s} head {g}")
        at += n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [4, 7, 9, 13, 20, 31, 60, 110])
@pytest.mark.parametrize("case", range(len(ROWS)))
def test_scores_of_any_size(case, size, dtype):
    """Five levels of scores up to 2^size, with many equal ones; rows of both signs."""
    rows, lens, hq, hkv = ROWS[case]
    gen = torch.Generator().manual_seed(600 + 10 * size + case)
    pool = Pool(list(lens), 16, hkv, 64, dtype, gen)
    k, q = torch.zeros(pool.kv[0].shape), torch.zeros(sum(rows), hq, 64)
    k[..., 5] = torch.randint(-2, 4, k.shape[:-1], generator=gen).float()
    q[..., 5] = 2.0 * torch.randint(0, 2, q.shape[:-1], generator=gen) - 1
    pool.kv[0].copy_(k.to(DT[dtype]))

    def bound(x, see, n, cols):
        X = float(x.abs().max())
        far = 2.0 ** (size - 2) > 150
        return (n + cols + 8 + (0 if far else 0.7 * (9 * X + 50) + 6 * (-(-n // 16) + 20))) * U
    compare(q.cuda().double(), k.cuda().double(), pool, rows, 2.0 ** (size - 2), bound, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(ROWS)))
def test_keys_of_the_types_lowest_value(case, dtype):
    """They weigh nothing beside others; a row that sees no others shares out among them."""
    rows, lens, hq, hkv = ROWS[case]
    gen = torch.Generator().manual_seed(700 + case)
    pool = Pool(list(lens), 16, hkv, 64, dtype, gen)
    k = torch.randint(-2, 3, pool.kv[0].shape, generator=gen).double()
    q = torch.randint(-2, 3, (sum(rows), hq, 64), generator=gen).double()
    k[..., 0], q[..., 0] = 0, 1
    masked = torch.rand(k.shape[:-1], generator=gen) < 0.5
    for s, L in enumerate(lens):  # the first keys all masked, every key of the last sequence
        for j in range(L if s == len(lens) - 1 else min(L, 45)):
            masked[int(pool.tables[s, j // 16]), j % 16] = True
    k[masked] = 0
    k[..., 0][masked] = torch.finfo(DT[dtype]).min
    pool.kv[0].copy_(k.to(DT[dtype]))
    lowest = float(torch.finfo(DT[dtype]).min)

    def bound(x, see, n, cols):
        X = float(x[x > lowest / 64].abs().max()) if bool((x > lowest / 64).any()) else 0.0
        return (n + cols + 8 + 0.7 * (9 * X + 50) + 6 * (-(-n // 16) + 20)) * U
    compare(q.cuda(), k.cuda(), pool, rows, 2.0 ** -4, bound, dtype)
