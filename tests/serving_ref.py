"""Plain 64-bit forms of the serving-step operators, sequence by sequence,
and the bounds that their tests use."""
from __future__ import annotations

import math

import torch

from paged_kv_gqa_02_gb300 import ops

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def cu(lens, device="cuda"):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)


def attend(q, k, v, see, scale):
    """One head: q [T][D], k and v [J][D], see [T][J] -> (out, sum of w |v|), float64."""
    s = (q @ k.T) * scale
    s = s.masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(top == -math.inf, 0.0, top)) * see
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return w @ v, w @ v.abs()


def bound(ref, weight, q, k, scale, n, dtype, out_dtype):
    """How far an element may be off.  A score is an fp32 dot product of D
    terms, off by D 2^-23 sum|q||k| at most (2^-23: the tensor cores may
    truncate), and so is its weight, relatively, with 2^-17 for the exponential
    and the two-part 16-bit probabilities; numerator and denominator both, hence
    twice.  Summing n terms in fp32 adds n 2^-23.  16-bit outputs add half a
    step of the result and half a step of each probability."""
    sabs = float((q.abs() @ k.abs().transpose(-1, -2)).max()) * scale if k.numel() else 0.0
    rel = 2 * (q.shape[-1] * 2.0 ** -23 * sabs + 2.0 ** -17) + n * 2.0 ** -23
    tol = weight * rel + 1e-30
    if out_dtype != "f32":
        half = torch.finfo(DT[out_dtype]).eps / 2
        tiny = torch.finfo(DT[out_dtype]).tiny * half * 2  # half a step of the subnormals
        tol = tol + half * (ref.abs() + weight) + tiny
    return tol


def reference(q, k, v, rows, keys_of, scale, dtype, out_dtype):
    """Expected output and bound of packed rows.  keys_of(s, g) gives the K, V
    (float64) and visibility of sequence s at kv head g."""
    hq, hkv = q.shape[1], k.shape[1]
    want = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.full_like(want, 1e-30)
    at = 0
    for s, n in enumerate(rows):
        for g in range(hkv if n else 0):
            kk, vv, see = keys_of(s, g, at)
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                qq = q[at:at + n, h].double()
                o, w = attend(qq, kk, vv, see, scale)
                want[at:at + n, h] = o
                tol[at:at + n, h] = bound(o, w, qq, kk, scale, kk.shape[0], dtype, out_dtype)
        at += n
    return want, tol


def prompt_ref(q, k, v, lens, scale, dtype, out_dtype):
    def keys_of(s, g, at):
        n = lens[s]
        see = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        return k[at:at + n, g].double(), v[at:at + n, g].double(), see
    return reference(q, k, v, lens, keys_of, scale, dtype, out_dtype)


def bits(mask, at, n):
    """Visibility [n][n] of the drafts at rows at..at+n-1 from their mask words."""
    word = mask[at:at + n].long()
    j = torch.arange(n, device=mask.device)
    return (word[:, j // 32] >> (j % 32)) & 1 == 1


def tree_ref(q, k, v, drafts, mask, k_cache, v_cache, tables, lens, scale, dtype, out_dtype):
    """k_cache, v_cache [pages][P][Hkv][D]; table entries outside the pool are skipped."""
    pages, page = k_cache.shape[:2]

    def keys_of(s, g, at):
        n, L = drafts[s], lens[s]
        pos = torch.arange(L, device=q.device)
        entry = tables[s].long()[pos // page]
        ok = (entry >= 0) & (entry < pages)
        entry, slot = entry[ok], (pos % page)[ok]
        kk = torch.cat([k_cache[entry, slot, g].double(), k[at:at + n, g].double()])
        vv = torch.cat([v_cache[entry, slot, g].double(), v[at:at + n, g].double()])
        see = torch.cat([torch.ones(n, len(entry), dtype=torch.bool, device=q.device), bits(mask, at, n)], 1)
        return kk, vv, see
    return reference(q, k, v, drafts, keys_of, scale, dtype, out_dtype)


def assert_close(got, want, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() / tol
    worst = int(over.argmax())
    assert float(over.max()) <= 1.0, (f"{what}: {float(over.max()):.2f} of the bound at {worst}: "
                                      f"{float(got.flatten()[worst])} for {float(want.flatten()[worst])}")


def random_mask(drafts, words, gen, empty=0.0):
    """Ancestor masks of random trees; with `empty`, that share of the rows sees nothing."""
    rows = []
    for n in drafts:
        seen = []
        for t in range(n):
            parent = int(torch.randint(0, t, (1,), generator=gen)) if t else -1
            b = (seen[parent] if t else 0) | (1 << t)
            seen.append(b)
            rows.append(0 if float(torch.rand(1, generator=gen)) < empty else b)
    out = torch.zeros(len(rows), words, dtype=torch.int64)
    for i, b in enumerate(rows):
        for w in range(words):
            x = (b >> (32 * w)) & 0xFFFFFFFF
            out[i, w] = x - (1 << 32) if x >= 1 << 31 else x
    return out.to(torch.int32).cuda()


class Pool:
    """A paged K/V pool with shuffled, disjoint tables and NaN wherever no token lies."""

    def __init__(self, lens, page, hkv, d, dtype, gen, spare=5, head_major=False, room=0):
        counts = [-(-n // page) for n in lens]
        self.pages, self.page, self.lens, self.hkv, self.d, self.dtype = sum(counts) + spare, page, lens, hkv, d, dtype
        self.blocks = max(max(counts) + room, 1)
        order = torch.randperm(self.pages, generator=gen).tolist()
        shape = (self.pages, hkv, page, d) if head_major else (self.pages, page, hkv, d)
        self.tables = torch.full((len(lens), self.blocks), -1, dtype=torch.int32)
        used = torch.zeros(self.pages, page, dtype=torch.bool)
        for s, n in enumerate(lens):
            for b in range(counts[s]):
                pg = order.pop()
                self.tables[s, b] = pg
                used[pg, :min(page, n - b * page)] = True
        self.tables = self.tables.cuda()
        self.context = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.k, self.v = (torch.randn(shape, generator=gen).to(DT[dtype]).cuda() for _ in range(2))
        # [pages][P][Hkv][D] views, whatever the storage order
        self.kv = [x.transpose(1, 2) if head_major else x for x in (self.k, self.v)]
        for x in self.kv:
            x[~used.cuda()] = float("nan")
        self.strides = (hkv * page * d, d, page * d) if head_major else (0, 0, 0)

    def params(self, hq, scale=None, out_dtype="f32", **kw):
        return ops.make_params(num_seqs=len(self.lens), num_q_heads=hq, num_kv_heads=self.hkv, head_dim=self.d,
                               page_size=self.page, num_pages=self.pages, max_blocks_per_seq=self.blocks,
                               max_context_len=self.blocks * self.page, scale=scale, dtype=self.dtype,
                               out_dtype=out_dtype, strides=self.strides, **kw)


# ---- the pages, on the host ------------------------------------------------------

class PageModel:
    """The bookkeeping's definition, one sequence after another."""

    def __init__(self, ref, tables, lens, page):
        self.ref, self.tables, self.lens, self.page = list(ref), [list(t) for t in tables], list(lens), page

    def up(self, n):
        return -(-n // self.page)

    def resize(self, new):
        old = list(self.ref)
        free = [i for i, r in enumerate(old) if r == 0]
        asked, pairs, short = 0, [], False
        for s, n in enumerate(new):
            pairs.append([-1, -1])
            if n < 0:
                continue
            L, table = self.lens[s], self.tables[s]
            edge = min(L, n)
            shared = edge % self.page != 0 and old[table[edge // self.page]] > 1
            need = max(0, self.up(n) - self.up(L)) + shared
            asked += need
            if need and asked > len(free):
                short = True
                continue
            mine = free[asked - need:asked]
            if shared:
                b = edge // self.page
                pairs[s] = [table[b], mine[0]]
                self.ref[table[b]] -= 1
                table[b] = mine.pop(0)
                self.ref[table[b]] += 1
            for b in range(self.up(n), self.up(L)):
                self.ref[table[b]] -= 1
                table[b] = -1
            for b in range(self.up(L), self.up(n)):
                table[b] = mine.pop(0)
                self.ref[table[b]] += 1
            self.lens[s] = n
        return pairs, short

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.lens[b] = self.lens[a]
            for i in range(self.up(self.lens[a])):
                self.tables[b][i] = self.tables[a][i]
                self.ref[self.tables[a][i]] += 1

    def compact(self, most):
        live = [i for i, r in enumerate(self.ref) if r]
        n = len(live)
        moves = list(zip([i for i in live if i >= n], [i for i in range(n) if not self.ref[i]]))[:most]
        to = dict(moves)
        for a, b in moves:
            self.ref[b], self.ref[a] = self.ref[a], 0
        for s, t in enumerate(self.tables):
            for i in range(self.up(self.lens[s])):
                t[i] = to.get(t[i], t[i])
        return [list(m) for m in moves] + [[-1, -1]] * (most - len(moves)), len(moves)
