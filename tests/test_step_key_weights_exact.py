"""pa_key_weights where every score is exact: q and k are whole numbers whose products and sums have at most 24 bits, in
any order, but more bits together than a narrower type's operands would keep.  What is left to be off is the softmax.

u = 2^-24, half a step of fp32.  X is the largest score in base 2, n the keys, C the columns of a kv head.
  the exponent of a term, s log2(e) scale - m: log2(e) is rounded (X u; the scale is a power of two), the product
    (X u), the difference (2 X u), and m + log2 l as one number ((X + 10) u, log2 l another 4 u of its 10)
  the denominator's terms the same but for the last: 4 X u.  A relative error is ln 2 times an exponent's, so
    0.7 (9 X + 50) u
  2^x is good to 2^-22, 4 u, above and below: 8 u; the reciprocal and the product with it: 3 u
  n terms below and C above, each addition u; a running maximum that changes rescales the sum, 6 u each: at most
    once for each tile of 16 keys and for each of 20 joins
Old weights, decay 1, add one more rounding of the sum."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from paged_kv_gqa_02_gb300 import ops
from serving_ref import DT, Pool, assert_close, cu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# largest q and k, dims of q that are not 0: every sum of products below 2^24.  fp32's k has more bits than tf32 keeps,
# fp16's more than bf16 does, bf16's all that it has
NUMBERS = {"f32": (511, 8191, 4), "f16": (1023, 2047, 6), "bf16": (255, 255, 64)}


@pytest.mark.parametrize("dtype", list(NUMBERS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,lens,hq,hkv", [
    ((1, 1, 1), (1, 64, 47), 4, 2),           # single tokens
    ((5, 1), (50, 64), 6, 1),                 # 30 columns
    ((20, 3, 1), (64, 33, 64), 6, 2),         # many columns
    ((64, 17), (64, 64), 3, 3)])              # whole prompts
def test_the_softmax_of_exact_scores(rows, lens, hq, hkv, d, dtype):
    qmax, kmax, some = NUMBERS[dtype]
    assert qmax * kmax * some < 2 ** 24
    gen = torch.Generator().manual_seed(500 + sum(rows) + d)
    pool = Pool(list(lens), 16, hkv, d, dtype, gen)
    k = torch.randint(-kmax, kmax + 1, pool.kv[0].shape, generator=gen)
    pool.kv[0].copy_(k.to(DT[dtype]))
    q = torch.randint(-qmax, qmax + 1, (sum(rows), hq, d), generator=gen)
    q[torch.rand(q.shape, generator=gen).argsort(-1) >= some] = 0
    group, scale = hq // hkv, 2.0 ** -(int(math.log2(qmax * kmax * some)) - 3)
    q, k = q.cuda().double(), k.cuda().double()
    weights = torch.rand(len(lens), hkv, pool.blocks * 16, generator=gen).cuda()
    want, tol, at = weights.double().clone(), torch.full(weights.shape, 1e-30, dtype=torch.float64, device="cuda"), 0
    for s, (n, L) in enumerate(zip(rows, lens)):
        spot = torch.arange(L, device="cuda")
        kk = k[pool.tables[s].long()[spot // 16], spot % 16]
        see = spot[None] <= torch.arange(L - n, L, device="cuda")[:, None]
        for g in range(hkv):
            score = torch.einsum("thd,jd->htj", q[at:at + n, g * group:(g + 1) * group], kk[:, g])
            assert float(score.abs().max()) < 2 ** 24
            X = float(score.abs().max()) * scale * math.log2(math.e)
            got = torch.softmax((score * scale).masked_fill(~see, -math.inf), 2).sum((0, 1))
            rel = (0.7 * (9 * X + 50) + 11 + L + n * group + 6 * (-(-L // 16) + 20)) * U
            old = want[s, g, :L].clone()
            old[L - n:] = 0
            want[s, g, :L] = got + old
            tol[s, g, :L] = rel * got + U * (got + old) + 1e-30
        at += n
    p, r = pool.params(hq, scale=scale), ops.make_rows(sum(rows), max(rows))
    got = ops.key_weights(p, r, q.to(DT[dtype]).contiguous(), cu(rows), pool.k, pool.tables, pool.context, weights)
    for s, L in enumerate(lens):
        assert_close(got[s, :, :L], want[s, :, :L], tol[s, :, :L], f"sequence {s}")
