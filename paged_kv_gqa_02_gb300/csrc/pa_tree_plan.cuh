// pa_tree_plan.cuh -- how a tree call's work is shared out, and the join of
// the pieces.
//
// A unit is (sequence, kv head, tile of `tu` drafts); its keys come in blocks
// of `kb`, first the history's, then the drafts' own.  Units are laid end to
// end, sequence by sequence and kv head by kv head, each as `start` positions
// and then, for a block, one position or, in a sequence whose units hold more
// than `tile` drafts, two: what starting and ending a unit and what a block
// cost beside one another.  The line is cut into n equal shares, one for each
// CTA; a block is the share's that holds its first position.  A unit inside one
// share is finished there; the pieces of the others are left in slots and
// joined in ascending CTA order.  A CTA leaves at most two pieces: one of a
// unit that began before its share (slot 2c) and one of a unit that begins in
// it (slot 2c + 1).  Shares have `min_share` positions at least, two where a
// block has two, so that none lies inside a unit without one of its blocks.
// The partition depends on the lengths and n alone, so results repeat bit for
// bit, and on the device only through n.
#pragma once

#include "pa_ptx.cuh"
#include "pa_serving.h"

#include <algorithm>

namespace pa {

namespace {  // each kernel's file has its own copy of the join

struct TreeShape {
    const int32_t* cu_lens;
    const int32_t* context_lens;
    int32_t num_seqs, total_rows, max_rows, Hkv, tu, tile, kb, start, min_share, n_ctas;
    int32_t cap;  // longest history: what a block table holds, 2^30 at most
};

struct TreeSeq {
    int row0, T, L;  // T = 0: no rows, or rows that the call refuses; L = 0 with a bad length
    bool bad_rows, bad_len;
    int units, nh, nd;   // tiles of a kv head; blocks of history and of drafts
    int width, cost;     // positions of a block and of a unit
};

// Sequence s from its lengths (no loads).
__device__ inline TreeSeq tree_seq_of(const TreeShape& a, int r0, int r1, int L) {
    TreeSeq q;
    q.row0 = r0;
    q.L = L;
    q.bad_rows = r0 < 0 || r1 < r0 || r1 > a.total_rows || r1 - r0 > a.max_rows;
    q.T = q.bad_rows ? 0 : r1 - r0;
    q.bad_len = L < 0 || L > a.cap;
    if (q.bad_len) q.L = 0;
    q.units = (q.T + a.tu - 1) / a.tu;
    q.nh = (q.L + a.kb - 1) / a.kb;
    q.nd = (q.T + a.kb - 1) / a.kb;
    q.width = q.T > a.tile ? 2 : 1;
    q.cost = q.T > 0 ? a.start + q.width * (q.nh + q.nd) : 0;
    return q;
}
__device__ inline TreeSeq tree_seq(const TreeShape& a, int s) {
    return tree_seq_of(a, a.cu_lens[s], a.cu_lens[s + 1], a.context_lens[s]);
}

__device__ inline int64_t tree_seq_cost(const TreeShape& a, const TreeSeq& q) {
    return int64_t(a.Hkv) * q.units * q.cost;
}

__device__ inline int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// CTAs that take part.
__device__ inline int tree_ctas(const TreeShape& a, int64_t total) {
    return int(min(int64_t(a.n_ctas), max(int64_t(1), total / a.min_share)));
}
// 64-bit division takes long; the usual operands fit 32 bits.
__device__ inline int64_t div_pos(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}
__device__ inline int64_t share_start(int64_t total, int n, int c) { return div_pos(total * c + n - 1, n); }
__device__ inline int share_owner(int64_t total, int n, int64_t p) { return int(div_pos(p * n, total)); }

// One CTA's piece of a unit.
struct TreeItem {
    int seq, g, row0;         // packed row of the tile's first draft
    int t0, n_rows;           // the tile's first draft, its drafts
    int T, L, nh, b0, b1;     // blocks [b0, b1) of nh + nd
    int slot;                 // -1: the whole unit
    int last;                 // of a unit's first piece: the CTA of its last one
    bool bad_len;
};

// A CTA's walk over its share, by one whole warp whose lanes hold the same
// state, but for the lengths of 32 sequences, one a lane: a call of up to 32
// sequences reads them once, in one round of loads.
struct TreeWalk {
    int64_t at, end;  // positions left
    int64_t seq_at;   // where the current sequence starts
    int64_t total;
    int s, cta, n;
    TreeSeq q;
    int base, lane_r0, lane_r1, lane_L;  // lengths of sequence base + lane

    __device__ inline void load(const TreeShape& a, int b) {
        base = b;
        const int i = b + int(threadIdx.x & 31);
        const bool in = i < a.num_seqs;
        lane_r0 = in ? a.cu_lens[i] : 0;
        lane_r1 = in ? a.cu_lens[i + 1] : 0;
        lane_L = in ? a.context_lens[i] : 0;
    }
    __device__ inline TreeSeq get(const TreeShape& a, int i) {
        const int l = i - base;
        return tree_seq_of(a, __shfl_sync(0xffffffffu, lane_r0, l), __shfl_sync(0xffffffffu, lane_r1, l),
                           __shfl_sync(0xffffffffu, lane_L, l));
    }
    __device__ inline int64_t lane_cost(const TreeShape& a) {  // 0 past the last sequence: it has no rows
        return tree_seq_cost(a, tree_seq_of(a, lane_r0, lane_r1, lane_L));
    }

    __device__ inline void start(const TreeShape& a, int c) {
        cta = c;
        load(a, 0);
        int64_t all = lane_cost(a);
#pragma unroll 4
        for (int i = 32 + int(threadIdx.x & 31); i < a.num_seqs; i += 32) all += tree_seq_cost(a, tree_seq(a, i));
        total = warp_sum64(all);
        n = tree_ctas(a, total);
        at = end = 0;
        if (c >= n || total == 0) return;
        at = share_start(total, n, c);
        end = share_start(total, n, c + 1);
        seq_at = 0;
        // the sequence that position `at` lies in, 32 at a time
#pragma unroll 1
        for (;;) {
            const int64_t own = lane_cost(a);
            int64_t upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (int(threadIdx.x & 31) >= o) upto += x;
            }
            const unsigned m = __ballot_sync(0xffffffffu, seq_at + upto > at);
            if (m) {
                const int l = __ffs(m) - 1;
                s = base + l;
                seq_at += __shfl_sync(0xffffffffu, upto - own, l);
                break;
            }
            seq_at += __shfl_sync(0xffffffffu, upto, 31);  // at < total: a later window has it
            load(a, base + 32);
        }
        q = get(a, s);
    }

    // The next piece; false at the share's end.
    __device__ inline bool next(const TreeShape& a, TreeItem& it) {
#pragma unroll 1
        while (at < end) {
#pragma unroll 1
            while (at >= seq_at + tree_seq_cost(a, q)) {  // at < end <= total: a later sequence has it
                seq_at += tree_seq_cost(a, q);
                if (++s - base == 32) load(a, s);
                q = get(a, s);
            }
            const int64_t in = at - seq_at;
            const int unit = int(div_pos(in, q.cost)), o = int(in - int64_t(unit) * q.cost);
            const int take = int(min(int64_t(q.cost - o), end - at));
            at += take;
            // blocks whose first position, start + width * b, is in [o, o + take)
            it.b0 = max(o - a.start + q.width - 1, 0) / q.width;
            it.b1 = max(o + take - a.start + q.width - 1, 0) / q.width;
            if (it.b0 >= it.b1) continue;  // of the unit's start only
            it.g = unit / q.units;
            it.seq = s;
            it.t0 = (unit - it.g * q.units) * a.tu;
            it.n_rows = min(a.tu, q.T - it.t0);
            it.row0 = q.row0 + it.t0;
            it.T = q.T;
            it.L = q.L;
            it.nh = q.nh;
            it.bad_len = q.bad_len;
            const bool first = it.b0 == 0, whole = first && it.b1 == q.nh + q.nd;
            it.slot = whole ? -1 : 2 * cta + (first ? 1 : 0);
            it.last = cta;
            if (first && !whole)  // the last block's first position
                it.last = share_owner(total, n, seq_at + int64_t(unit) * q.cost + a.start + q.width * (q.nh + q.nd - 1));
            return true;
        }
        return false;
    }
};

// Lengths that a call refuses are flagged once, by CTA 0.
__device__ inline void tree_flag_lengths(const TreeShape& a, uint32_t* status) {
    for (int s = threadIdx.x; s < a.num_seqs; s += blockDim.x) {
        const TreeSeq q = tree_seq(a, s);
        if (q.bad_rows || q.bad_len) flag(status, PA_DEV_BAD_LEN);
    }
}

// A slot holds, for each of a unit's `rows` distributions (draft * G + head),
// the base-2 running max and the sum, then the accumulators.
__host__ __device__ inline int64_t slot_floats(int rows, int D) { return int64_t(rows) * (D + 2); }

// The workspace: two slots for each CTA, then for each CTA the unit to join that
// begins in its share (one at most): its first packed row, kv head, drafts (0:
// none), and the CTA of its last piece.
__host__ __device__ inline size_t tree_workspace_bytes(int rows, int D, int n_ctas) {
    return (size_t(n_ctas) * (2 * slot_floats(rows, D) * sizeof(float) + sizeof(int4)) + 255) & ~size_t(255);
}
__device__ inline int4* tree_joins(void* workspace, int rows, int D, int n_ctas) {
    return reinterpret_cast<int4*>(static_cast<float*>(workspace) + 2 * slot_floats(rows, D) * n_ctas);
}
__device__ inline bool begins(const TreeItem& it) { return it.slot >= 0 && (it.slot & 1); }
__device__ inline int4 join_of(const TreeItem& it) { return make_int4(it.row0, it.g, it.n_rows, it.last); }

template <typename T> __device__ inline T from_f32(float x);
template <> __device__ inline float from_f32<float>(float x) { return x; }
template <> __device__ inline __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ inline __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// The join, launched with programmatic dependent launch behind the pieces'
// kernel, which leaves it a list of what to join.  CTAs of eight warps over a
// unit's distributions, `per` for each warp one after the other.  Pieces are
// taken in ascending CTA order, kP at a time in flight, against a running max.
// A small call has many pieces for each of few distributions and waits for its
// loads: sixteen in flight, a distribution a warp.  A large one has two or three
// pieces for each of many and is bound by its instructions (36 us with sixteen
// steps for each, 64 rows x 8, 64 heads): four in flight, two distributions a
// warp.
template <typename TOut, int D, int kP>
__global__ void __launch_bounds__(256)
    tree_join(float* slots, TOut* out, int Hq, int G, int rows, int per, int n_ctas) {
    constexpr int kV = D / 32;  // dims of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait_primary();
    // the blockIdx.x-th entry of the list that has something to join
    __shared__ int count[8], found;
    const int4* list = tree_joins(slots, rows, D, n_ctas);
    int left = blockIdx.x;
    if (threadIdx.x == 0) found = -1;
#pragma unroll 1
    for (int base = 0; base < n_ctas; base += 256) {
        const int i = base + int(threadIdx.x);
        const bool has = i < n_ctas && list[i].z > 0;
        const unsigned m = __ballot_sync(0xffffffffu, has);
        if (lane == 0) count[warp] = __popc(m);
        __syncthreads();
        int at = __popc(m & ((1u << lane) - 1u)), all = 0;
        for (int w = 0; w < 8; ++w) {
            at += w < warp ? count[w] : 0;
            all += count[w];
        }
        if (has && at == left) found = i;
        left -= all;
        __syncthreads();
    }
    if (found < 0) return;
    const int4 u = list[found];
    const int valid = u.z * G, c0 = found, c1 = u.w;
    const int64_t size = slot_floats(rows, D);
    // a piece's slot: the unit's first CTA left it in its second
    const float* first = slots + size * (2 * c0 + 1);
    const float* later = slots + size * (2 * c0);  // + 2 * size for each CTA on
#pragma unroll 1
    for (int k = 0; k < per; ++k) {
        const int r = (int(blockIdx.y) * 8 + warp) * per + k;
        if (r >= valid) return;
        float acc[kV], m_run = -INFINITY, l_run = 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v) acc[v] = 0.f;
#pragma unroll 1
        for (int c = c0; c <= c1; c += kP) {
            const int np = min(kP, c1 - c + 1);
            float2 ml = make_float2(-INFINITY, 0.f);  // of piece `lane`
            auto slot_of = [&](int i) { return c + i == c0 ? first : later + 2 * size * (c + i - c0); };
            if (lane < np) ml = *reinterpret_cast<const float2*>(slot_of(lane) + 2 * r);
            float x[kP][kV];
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                if (i >= np) break;
                const float* p = slot_of(i) + 2 * rows + int64_t(r) * D + lane * kV;
                if constexpr (kV == 4)
                    *reinterpret_cast<float4*>(x[i]) = *reinterpret_cast<const float4*>(p);
                else
                    *reinterpret_cast<float2*>(x[i]) = *reinterpret_cast<const float2*>(p);
            }
            const float m_new = fmaxf(m_run, warp_max(ml.x));
            const float base = m_new == -INFINITY ? 0.f : m_new;
            const float old = ex2(m_run - base);
            m_run = m_new;
            // a piece with nothing visible has max -inf and sum 0: weight 0.  With
            // a sum that is not 0 its scores were NaN, which the max drops.
            const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - base);
            l_run *= old;
#pragma unroll
            for (int v = 0; v < kV; ++v) acc[v] *= old;
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                if (i >= np) break;
                const float wi = __shfl_sync(0xffffffffu, w, i), li = __shfl_sync(0xffffffffu, ml.y, i);
                if (wi != 0.f) {
                    l_run = fmaf(wi, li, l_run);
#pragma unroll
                    for (int v = 0; v < kV; ++v) acc[v] = fmaf(wi, x[i][v], acc[v]);
                }
            }
        }
        const int t = r / G;
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
        TOut y[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) y[v] = from_f32<TOut>(acc[v] * inv);
        TOut* o = out + (int64_t(u.x + t) * Hq + u.y * G + (r - t * G)) * D + lane * kV;
        if constexpr (sizeof(y) == 16)
            *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(y);
        else if constexpr (sizeof(y) == 8)
            *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(y);
        else
            *reinterpret_cast<uint32_t*>(o) = *reinterpret_cast<const uint32_t*>(y);
    }
}
// Launches it: one distribution a warp while that makes no more CTAs with work
// than run at once, two otherwise.
template <typename TOut, int D>
inline cudaError_t launch_join(const TreeShape& a, const PackedAttn& p, int rows, cudaStream_t st) {
    const int64_t units = int64_t(a.Hkv) * (a.total_rows / a.tu + std::min(a.num_seqs, a.total_rows));
    const int G = p.Hq / p.Hkv, most = std::min(a.tu, a.max_rows) * G;  // a unit's distributions
    const int per = units * ((most + 7) / 8) <= 152 * 4 ? 1 : 2;
    return launch_pdl(per == 1 ? tree_join<TOut, D, 16> : tree_join<TOut, D, 4>,
                      dim3(unsigned(std::min(units, int64_t(a.n_ctas))), (most + 8 * per - 1) / (8 * per)), dim3(256), 0, st,
                      static_cast<float*>(p.workspace), static_cast<TOut*>(p.out), p.Hq, G, rows, per, a.n_ctas);
}

}  // namespace

}  // namespace pa
