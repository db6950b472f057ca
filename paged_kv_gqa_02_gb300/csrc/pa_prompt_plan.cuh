// pa_prompt_plan.cuh -- a prompt call's units of work, numbered.
//
// A unit is (sequence, kv head, tile of `tu` rows); its keys are the sequence's
// rows up to its own, in blocks of `kb`.  Up to 32 sequences: units in descending
// order of their keys, by level (the tile of rows, from the last), then
// sequence, then kv head.  More: by sequence, then level from the last, then kv
// head, as finding a level would mean counting all sequences again for each unit.
#pragma once

#include "pa_serving.h"
#include "pa_tree_plan.cuh"

#include <algorithm>

namespace pa {

namespace {

struct PromptShape {
    const int32_t* cu_lens;
    int32_t num_seqs, total_rows, max_rows, Hkv, tu, kb;
    int32_t n_units;  // of the longest sequence that there can be, per kv head
};

inline PromptShape prompt_shape(const PackedAttn& a, int tu, int kb) {
    return {a.r.cu_lens, a.r.num_seqs, a.r.total_rows, a.r.max_rows, a.Hkv, tu, kb, (a.r.max_rows + tu - 1) / tu};
}
// Numbers that there can be: a sequence's last unit may be partly filled.
inline int64_t prompt_numbers(const PromptShape& a) {
    return std::min(int64_t(a.Hkv) * a.num_seqs * a.n_units, int64_t(a.Hkv) * (a.total_rows / a.tu + a.num_seqs));
}

// Finds units by their numbers; by one whole warp.
struct PromptUnits {
    int base, first;  // the window of 32 sequences at hand; units of those before it
    int lane_n;       // units of sequence base + lane
    __device__ inline void load(const PromptShape& a, int b) {
        const int s = b + int(threadIdx.x & 31);
        base = b;
        lane_n = 0;
        if (s < a.num_seqs) {
            const int r0 = a.cu_lens[s], r1 = a.cu_lens[s + 1];
            if (r0 >= 0 && r1 >= r0 && r1 <= a.total_rows && r1 - r0 <= a.max_rows)
                lane_n = (r1 - r0 + a.tu - 1) / a.tu;
        }
    }
    __device__ inline void start(const PromptShape& a) {
        first = 0;
        load(a, 0);
    }
    static __device__ inline int warp_add(int n) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        return n;
    }
    // Unit number i; false where there are not so many.
    __device__ inline bool get(const PromptShape& a, int i, TreeItem& it) {
        const int k = i / a.Hkv;
        int level;
        if (a.num_seqs <= 32) {
            if (k >= warp_add(lane_n)) return false;
            int lo = 0, hi = a.n_units - 1;  // the highest level with more than k units at and above it
#pragma unroll 1
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (warp_add(max(0, lane_n - mid)) > k)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            level = lo;
            int rank = k - warp_add(max(0, lane_n - lo - 1));  // among the sequences that reach this level
            unsigned m = __ballot_sync(0xffffffffu, lane_n > lo);
#pragma unroll 1
            for (; rank > 0; --rank) m &= m - 1;
            it.seq = __ffs(m) - 1;
        } else {
            if (k < first) start(a);  // numbers mostly rise
            int all;
#pragma unroll 1
            while (k >= first + (all = warp_add(lane_n))) {
                if (base + 32 >= a.num_seqs) return false;
                first += all;
                load(a, base + 32);
            }
            int upto = lane_n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (int(threadIdx.x & 31) >= o) upto += y;
            }
            const int l = __ffs(__ballot_sync(0xffffffffu, first + upto > k)) - 1;
            it.seq = base + l;
            level = first + __shfl_sync(0xffffffffu, upto, l) - 1 - k;  // the sequence's last unit first
        }
        const int r0 = a.cu_lens[it.seq];
        it.g = i - k * a.Hkv;
        it.T = a.cu_lens[it.seq + 1] - r0;
        it.t0 = level * a.tu;
        it.n_rows = min(a.tu, it.T - it.t0);
        it.row0 = r0 + it.t0;
        it.L = it.nh = it.b0 = 0;
        it.b1 = (it.t0 + it.n_rows + a.kb - 1) / a.kb;
        it.slot = -1;
        it.last = 0;
        it.bad_len = false;
        return true;
    }
};

}  // namespace

}  // namespace pa
