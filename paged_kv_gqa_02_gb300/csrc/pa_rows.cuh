// pa_rows.cuh -- which sequence a packed row belongs to, and whether the
// sequences' rows are in range (serving-step kernels).
#pragma once

#include "pa_common.cuh"

namespace pa {

__device__ inline bool bad_rows(int r0, int r1, int total_rows, int max_rows) {
    return r0 < 0 || r1 < r0 || r1 > total_rows || r1 - r0 > max_rows;
}

// Flags sequences whose rows are out of range: one CTA of a grid does it, as a
// sequence without rows of its own is seen by nobody else.
__device__ inline void flag_bad_rows(const int32_t* cu_lens, int num_seqs, int total_rows, int max_rows,
                                     uint32_t* dev_status) {
    for (int s = threadIdx.x; s < num_seqs; s += blockDim.x)
        if (bad_rows(cu_lens[s], cu_lens[s + 1], total_rows, max_rows)) flag(dev_status, PA_DEV_BAD_LEN);
}

// The number of sequence ends at or before the row, 32 probes at a time (whole
// warp): its sequence, or num_seqs behind the last one.
__device__ inline int seq_of_row(const int32_t* cu_lens, int num_seqs, int row, int lane) {
    int lo = 0, hi = num_seqs;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + step * (lane + 1) - 1;  // the last of each of 32 runs
        const int k = __popc(__ballot_sync(0xffffffffu, at < hi && cu_lens[at + 1] <= row));
        lo = min(lo + step * k, hi);
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

}  // namespace pa
