// pa_checks.h -- what the serving-step entry points check of their arguments
// on the host, before any device access (internal to the library).
#pragma once

#include <math.h>

#include "pa_serving.h"

namespace {  // each file of entry points has its own copy

constexpr int kRefSms = 152;         // SMs that a deterministic call is laid out for
constexpr int kMaxTreeRows = 1024;   // drafts of one sequence
constexpr int kMaxRows = 1 << 30;    // packed rows: sums with a tile stay in 32 bits
constexpr int64_t kMaxHistory = 1 << 30;  // tokens before a tree, for the same reason

inline int elt_bytes(pa_dtype d) { return d == PA_F32 ? 4 : 2; }
inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool known_dtype(pa_dtype d) { return d >= PA_F32 && d <= PA_BF16; }

inline int device_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return kRefSms;
    return n;
}

inline pa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// Heads, dtypes and scale of an attention call.
inline pa_status check_heads(const pa_params* p) {
    if (p->num_seqs < 1 || p->num_q_heads < 1 || p->num_kv_heads < 1) return PA_ERR_SHAPE;
    if (p->num_seqs > 65535 || p->num_kv_heads > 65535) return PA_ERR_SHAPE;
    if (p->num_q_heads % p->num_kv_heads != 0) return PA_ERR_SHAPE;
    if (!known_dtype(p->q_dtype) || !known_dtype(p->kv_dtype) || !known_dtype(p->out_dtype)) return PA_ERR_DTYPE;
    if (p->num_q_heads / p->num_kv_heads > pa::kMaxGroup) return PA_ERR_UNSUPPORTED;
    if (p->head_dim != 64 && p->head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (p->q_dtype != p->kv_dtype || (p->out_dtype != PA_F32 && p->out_dtype != p->q_dtype))
        return PA_ERR_UNSUPPORTED;
    if (!isfinite(p->scale) || !(p->scale > 0.f)) return PA_ERR_SHAPE;
    if (p->debug_timeout != 0 && p->debug_timeout != 1) return PA_ERR_SHAPE;
    return PA_OK;
}

// The pool's geometry, as pa_decode takes it.
inline pa_status check_cache(const pa_params* p, pa::CacheArgs* c) {
    if (p->num_seqs < 1 || p->num_seqs > 65535 || p->num_kv_heads < 1 || p->num_kv_heads > 65535)
        return PA_ERR_SHAPE;
    if (!known_dtype(p->kv_dtype)) return PA_ERR_DTYPE;
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return PA_ERR_UNSUPPORTED;
    if (p->page_size != 16 && p->page_size != 32) return PA_ERR_UNSUPPORTED;
    if (p->num_pages < 1 || p->max_blocks_per_seq < 1) return PA_ERR_SHAPE;
    const int64_t D = p->head_dim;
    c->head_stride = p->head_stride ? p->head_stride : D;
    c->token_stride = p->token_stride ? p->token_stride : p->num_kv_heads * c->head_stride;
    c->page_stride = p->page_stride ? p->page_stride : p->page_size * c->token_stride;
    if (c->head_stride < 0 || c->token_stride < 0 || c->page_stride < 0) return PA_ERR_SHAPE;
    const int eb = elt_bytes(p->kv_dtype);
    if ((c->head_stride * eb) % 16 || (c->token_stride * eb) % 16 || (c->page_stride * eb) % 16)
        return PA_ERR_ALIGN;
    c->page_size = p->page_size;
    c->num_pages = p->num_pages;
    c->max_blocks = p->max_blocks_per_seq;
    return PA_OK;
}

// Packed rows: strides hold a row of heads each and keep 16-byte alignment.
inline pa_status check_rows(const pa_params* p, const pa_rows* r, pa::RowArgs* a) {
    if (r->total_rows < 0 || r->max_rows < 0 || (r->total_rows > 0 && r->max_rows < 1)) return PA_ERR_SHAPE;
    if (r->source_rows < 0 || r->mask_words < 0) return PA_ERR_SHAPE;
    if (r->total_rows > kMaxRows) return PA_ERR_UNSUPPORTED;
    const int64_t D = p->head_dim, nq = D * p->num_q_heads, nk = D * p->num_kv_heads;
    a->num_seqs = p->num_seqs;
    a->total_rows = r->total_rows;
    a->max_rows = r->max_rows < r->total_rows ? r->max_rows : r->total_rows;
    a->q_stride = r->q_stride ? r->q_stride : nq;
    a->k_stride = r->k_stride ? r->k_stride : nk;
    a->v_stride = r->v_stride ? r->v_stride : nk;
    if ((r->q_stride && r->q_stride < nq) || a->k_stride < nk || a->v_stride < nk) return PA_ERR_SHAPE;
    const int eb = elt_bytes(p->kv_dtype);
    if ((a->q_stride * eb) % 16 || (a->k_stride * eb) % 16 || (a->v_stride * eb) % 16) return PA_ERR_ALIGN;
    return PA_OK;
}

inline int share_ctas(const pa_params* p) { return p->deterministic ? kRefSms : device_sms(); }

}  // namespace
