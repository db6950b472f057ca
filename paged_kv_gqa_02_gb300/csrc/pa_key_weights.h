// pa_key_weights.h -- what the key weights' kernels share (internal to the
// library).
#pragma once

#include "pa_rows.cuh"
#include "pa_serving.h"

namespace pa {

constexpr float kLowestScore = -3.402823466e38f;  // a running maximum before the first score

struct KwArgs {
    const void* q;
    const void* k;
    const int32_t* cu_lens;
    const int32_t* block_tables;
    const int32_t* context_lens;
    float* weights;
    float2* stats;  // [total_rows][Hq]: a column's largest score and the reciprocal of its sum
    float* scores;  // few columns: [num_seqs][Hkv][max_len][width]
    float2* pieces; // few columns: [num_seqs][Hkv][max_pieces][width], largest score and sum of a warp's part
    int32_t width;  // of a key's scores, the columns rounded up to even
    int64_t max_pieces;
    uint32_t* dev_status;
    int64_t q_stride, page_stride, token_stride, head_stride;
    int64_t slots;  // of a block table
    int32_t num_seqs, total_rows, max_rows, num_pages, max_blocks, page_size, page_shift;
    int32_t Hq, Hkv, G, max_len;
    float scale_log2, decay;
    int32_t debug_timeout;
};

struct KwSeq {
    int row0, T, L;
    bool bad;
};
__device__ inline KwSeq kw_seq(const KwArgs& a, int s) {
    KwSeq q;
    q.row0 = a.cu_lens[s];
    const int r1 = a.cu_lens[s + 1];
    q.L = a.context_lens[s];
    q.T = r1 - q.row0;
    q.bad = bad_rows(q.row0, r1, a.total_rows, a.max_rows) || q.L < q.T || q.L > a.max_len;
    if (q.bad) q.T = 0;
    return q;
}

// 1 / l, and 0 for a column that saw nothing (a NaN stays one).
__device__ inline float kw_reciprocal(float l) { return l == 0.f ? 0.f : 1.f / l; }

__device__ inline void kw_join(float& m, float& l, float m2, float l2) {
    const float top = fmaxf(m, m2);
    l = l * ex2(m - top) + l2 * ex2(m2 - top);
    m = top;
}

// Many columns of a 16-bit type, on the tensor cores; p.k is a cache of
// c.num_pages pages.  `parts` is key_weights_tc_parts bytes.
size_t key_weights_tc_parts(int n_ctas);
cudaError_t launch_key_weights_tc(const KwArgs& a, pa_dtype dt, int D, int n_ctas, void* parts, cudaStream_t st);

}  // namespace pa
