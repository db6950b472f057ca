// pa_serving.h -- launchers of the serving-step kernels (internal to the
// library): prompt and tree attention, the K/V store and the page operations.
#pragma once

#include "pa_common.cuh"
#include "paged_gqa_serving.h"

namespace pa {

// Packed rows with their strides resolved (elements).
struct RowArgs {
    const int32_t* cu_lens;
    int32_t num_seqs, total_rows, max_rows;
    int64_t q_stride, k_stride, v_stride;
};

// The paged cache with its strides resolved (elements).
struct CacheArgs {
    const void* k;
    const void* v;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t page_size, num_pages, max_blocks;
    int64_t page_stride, token_stride, head_stride;
};

// Attention of packed rows over themselves (prompt) or over a paged history
// and themselves under a mask (tree: tree_mask set).
struct PackedAttn {
    RowArgs r;
    const void* q;
    const void* k;
    const void* v;
    void* out;
    pa_dtype dtype, out_dtype;
    int32_t Hq, Hkv, D;
    float scale_log2;  // > 0
    uint32_t* dev_status;
    int32_t debug_timeout;
    // tree only
    const uint32_t* tree_mask;  // nullptr: prompt
    int32_t mask_words;
    int32_t max_history;  // what a block table holds, 2^30 at most
    CacheArgs c;
    int32_t n_ctas;
    void* workspace;
};

struct StoreCall {
    RowArgs r;
    const void* k;
    const void* v;
    const int32_t* row_index;
    int32_t source_rows, Hkv, D, elt_bytes;
    CacheArgs c;  // k, v written
    uint32_t* dev_status;
};
cudaError_t launch_store(const StoreCall& c, cudaStream_t st);

// fp32 on the CUDA cores; 16-bit types on the tensor cores.
cudaError_t launch_packed_f32(const PackedAttn& a, cudaStream_t st);
size_t tree_f32_workspace_bytes(int D, int n_ctas);
cudaError_t launch_packed_tc(const PackedAttn& a, cudaStream_t st);
size_t tree_tc_workspace_bytes(int D, int n_ctas);

struct PagesCall {
    int32_t* refcounts;
    int32_t* block_tables;
    int32_t* context_lens;
    int32_t num_seqs, num_pages, max_blocks, page_size;
    void* workspace;
    uint32_t* dev_status;
};
constexpr int kMaxPoolPages = 1 << 23;  // pages the bookkeeping calls take
size_t pages_workspace_bytes(int num_seqs, int num_pages);
cudaError_t launch_pages_resize(const PagesCall& c, const int32_t* new_lens, int32_t* pairs, cudaStream_t st);
cudaError_t launch_pages_fork(const PagesCall& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t st);
cudaError_t launch_pages_compact(const PagesCall& c, int32_t* pairs, int max_moves, int32_t* num_moves,
                                 cudaStream_t st);
cudaError_t launch_pages_copy(const CacheArgs& c, int Hkv, int D, int elt_bytes, const int32_t* pairs, int n,
                              uint32_t* dev_status, cudaStream_t st);

// Rotation, draft verification, key weights and eviction.
struct RotateCall {
    RowArgs r;
    pa_rope t;  // resolved: axes >= 1, strides in elements
    const void* q;
    const void* k;
    const void* v;
    const void* q_weight;
    const void* k_weight;
    void* q_out;
    void* k_out;
    const float* table;
    const int32_t* positions;
    pa_dtype dtype;
    int32_t Hq, Hkv, D;
    CacheArgs c;  // k == nullptr: no store
    uint32_t* dev_status;
};
cudaError_t launch_rotate(const RotateCall& c, cudaStream_t st);

struct VerifyCall {
    const int32_t* cu_lens;
    const void* logits;
    const void* draft;  // nullptr: certain drafts
    const int32_t* tokens;
    const int32_t* parents;
    const float* temperature;
    const float* uniform;
    const float* noise;
    const int32_t* context_lens;
    int32_t* accepted;
    int32_t* accepted_cu;
    int32_t* next_tokens;
    int32_t* new_lens;
    int64_t logits_stride, draft_stride;
    int32_t num_seqs, total_rows, max_rows, vocab;
    pa_dtype dtype;
    uint32_t* dev_status;
    int32_t debug_timeout;
};
cudaError_t launch_verify(const VerifyCall& c, cudaStream_t st);

struct KeyWeightsCall {
    RowArgs r;
    const void* q;
    CacheArgs c;  // v unused
    float* weights;
    pa_dtype dtype;
    int32_t Hq, Hkv, D;
    int32_t max_len;  // longest context taken
    int32_t n_ctas;
    float scale_log2, decay;
    void* workspace;
    uint32_t* dev_status;
    int32_t debug_timeout;
};
size_t key_weights_workspace_bytes(const KeyWeightsCall& c);
cudaError_t launch_key_weights(const KeyWeightsCall& c, cudaStream_t st);

struct EvictCall {
    CacheArgs c;  // k, v written
    const int32_t* refcounts;
    const float* weights;
    const int32_t* keep_lens;
    float* weights_out;
    int32_t* kept;
    int32_t* new_lens;
    int32_t num_seqs, Hkv, D, elt_bytes, first, recent;
    uint32_t* dev_status;
};
constexpr int64_t kMaxEvictSlots = 1 << 22;  // slots of a block table that pa_evict takes
cudaError_t launch_evict(const EvictCall& c, cudaStream_t st);

// A launch that may start while the kernel before it drains; its kernel waits
// (griddepcontrol.wait) before it touches global memory.
template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*k)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace pa
