"""Prompt and tree attention with scores of large size, up to those whose steps in
fp32 are whole powers of two of a weight.  All dims of a row of q are one power
of two and all of a key one small integer (times a power of two), so that scores
are exact in fp32 and two of them are equal or far apart: the result is the mean
of V over the keys with the largest score.  What is left of the bound is that of
the sums and of the rounding."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gqa_02_gb300 import build, ops
import serving_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]
# exponents of q's and of k's power of two: with 64 dims, a scale of 1/8 and integers of up to 8 bits a score is up
# to 2^(3 + 8 + both) in size
POWERS = {"f16": ((0, 0), (5, 2), (12, 2), (15, 0), (15, 4), (15, 7)), "bf16": ((0, 0), (8, 2), (16, 0), (20, 3), (40, 20), (50, 50))}
POWERS["f32"] = POWERS["bf16"]
SCALE = 0.125


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    ops.load()


def integers(gen, n, kind):
    """One integer a key: any, rising (the max moves with every tile), or negative."""
    c = torch.randint(-255, 256, (n,), generator=gen)
    return {"any": c, "rising": c.sort().values, "negative": -c.abs() - 1}[kind].double().clamp(-255, 255)


def rows(c, power, hkv, d, dtype):
    return (c * 2.0 ** power)[:, None, None].expand(-1, hkv, d).to(ref.DT[dtype]).contiguous().cuda()


def expected(k, v, c, see, hq, out_dtype):
    """From the integers: the mean of V over the largest that each row sees ([T][J] `see`)."""
    s = torch.where(see, c[None].to(see.device), -1e9)
    w = (see & (s == s.amax(-1, keepdim=True))).double()
    w = w / w.sum(-1, keepdim=True).clamp(min=1)
    want = torch.stack([w @ v[:, h // (hq // v.shape[1])].double() for h in range(hq)], 1)
    size = torch.stack([w @ v[:, h // (hq // v.shape[1])].double().abs() for h in range(hq)], 1)
    none = torch.zeros(1, 1, dtype=torch.float64, device=v.device)  # scores are exact
    return want, ref.bound(want, size, none, none, 1.0, see.shape[1], None, out_dtype)


@pytest.mark.parametrize("kind", ("any", "rising", "negative"))
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_prompt_wide_scores(dtype, out_dtype, kind):
    gen = torch.Generator().manual_seed(11)
    for hq, hkv, n in ((4, 2, 700), (16, 8, 600)):
        c = integers(gen, n, kind)
        v = torch.randn((n, hkv, 64), generator=gen).to(ref.DT[dtype]).cuda()
        p = ops.prompt_params(num_seqs=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=64, scale=SCALE, dtype=dtype,
                              out_dtype=out_dtype)
        see = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for a, b in POWERS[dtype]:
            k = rows(c, b, hkv, 64, dtype)
            q = rows(torch.ones(n, dtype=torch.float64), a, hq, 64, dtype)
            if (a, b) == (0, 0):  # neighbours are 8 apart here, not further: the plain form
                want, tol = ref.prompt_ref(q, k, v, [n], SCALE, dtype, out_dtype)
            else:
                want, tol = expected(k, v, c, see, hq, out_dtype)
            out = ops.prompt(p, ops.make_rows(n, n), q, k, v, ref.cu([n]))
            ref.assert_close(out, want, tol, f"2^{a} 2^{b} {hq}/{hkv}")


@pytest.mark.parametrize("kind", ("any", "rising", "negative"))
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_tree_wide_scores(dtype, out_dtype, kind):
    """A history over many CTAs, and short ones of one or two."""
    gen = torch.Generator().manual_seed(12)
    hq, hkv, page = 8, 2, 16
    lens, drafts = [3000, 200, 0, 500], [9, 20, 7, 70]
    pool = ref.Pool(lens, page, hkv, 64, dtype, gen)
    total = sum(drafts)
    v = torch.randn((total, hkv, 64), generator=gen).to(ref.DT[dtype]).cuda()
    mask = ref.random_mask(drafts, 3, gen)
    p, r = pool.params(hq, out_dtype=out_dtype, scale=SCALE), ops.make_rows(total, max(drafts))
    whole = [integers(gen, n + m, kind) for n, m in zip(lens, drafts)]
    for a, b in POWERS[dtype][1:]:
        q = rows(torch.ones(total, dtype=torch.float64), a, hq, 64, dtype)
        k = rows(torch.cat([c[n:] for c, n in zip(whole, lens)]), b, hkv, 64, dtype)
        for s, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            pool.kv[0][pool.tables[s].long()[pos // page], pos % page] = rows(whole[s][:n], b, hkv, 64, dtype)
        out = ops.tree(p, r, q, k, v, ref.cu(drafts), mask, pool.k, pool.v, pool.tables, pool.context)
        at = 0
        for s, (n, m) in enumerate(zip(lens, drafts)):
            pos = torch.arange(n, device="cuda")
            vv = torch.cat([pool.kv[1][pool.tables[s].long()[pos // page], pos % page], v[at:at + m]])
            see = torch.cat([torch.ones(m, n, dtype=torch.bool, device="cuda"), ref.bits(mask, at, m)], 1)
            want, tol = expected(None, vv, whole[s].cuda(), see, hq, out_dtype)
            ref.assert_close(out[at:at + m], want, tol, f"2^{a} 2^{b} sequence {s}")
            at += m
