// pa_serving_api.cu -- the extern "C" entry points of paged_gqa_serving.h:
// host-side validation (before any device access) and dispatch.  No entry
// point allocates memory.
#include <math.h>
#include <string.h>

#include "pa_serving.h"

#define PA_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr int kRefSms = 152;         // SMs that a deterministic call is laid out for
constexpr int kMaxTreeRows = 1024;   // drafts of one sequence
constexpr int kMaxRows = 1 << 30;    // packed rows: sums with a tile stay in 32 bits
constexpr int64_t kMaxHistory = 1 << 30;  // tokens before a tree, for the same reason

int elt_bytes(pa_dtype d) { return d == PA_F32 ? 4 : 2; }
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known_dtype(pa_dtype d) { return d >= PA_F32 && d <= PA_BF16; }

int device_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return kRefSms;
    return n;
}

pa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// Heads, dtypes and scale of an attention call.
pa_status check_heads(const pa_params* p) {
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
pa_status check_cache(const pa_params* p, pa::CacheArgs* c) {
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
pa_status check_rows(const pa_params* p, const pa_rows* r, pa::RowArgs* a) {
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

int share_ctas(const pa_params* p) { return p->deterministic ? kRefSms : device_sms(); }

pa_status check_tree(const pa_params* p, const pa_rows* r, pa::PackedAttn* a) {
    if (!p || !r) return PA_ERR_NULL;
    pa_status st = check_heads(p);
    if (st != PA_OK) return st;
    if ((st = check_cache(p, &a->c)) != PA_OK) return st;
    if ((st = check_rows(p, r, &a->r)) != PA_OK) return st;
    if (p->deterministic != 0 && p->deterministic != 1) return PA_ERR_SHAPE;
    if (p->num_splits != 0 || p->sliding_window != 0 || p->decode_q_rows > 1) return PA_ERR_UNSUPPORTED;
    if (a->r.max_rows > kMaxTreeRows) return PA_ERR_UNSUPPORTED;
    const int words = (a->r.max_rows + 31) / 32;
    a->mask_words = r->mask_words ? r->mask_words : int((int64_t(r->max_rows) + 31) / 32);
    if (a->mask_words < words) return PA_ERR_SHAPE;
    const int64_t cap = int64_t(p->max_blocks_per_seq) * p->page_size;
    a->max_history = int(cap < kMaxHistory ? cap : kMaxHistory);
    a->n_ctas = share_ctas(p);
    return PA_OK;
}

size_t tree_bytes(const pa_params* p, int n_ctas) {
    return p->kv_dtype == PA_F32 ? pa::tree_f32_workspace_bytes(p->head_dim, n_ctas)
                                 : pa::tree_tc_workspace_bytes(p->head_dim, n_ctas);
}

void fill_heads(const pa_params* p, pa::PackedAttn* a) {
    a->dtype = p->q_dtype;
    a->out_dtype = p->out_dtype;
    a->Hq = p->num_q_heads;
    a->Hkv = p->num_kv_heads;
    a->D = p->head_dim;
    a->scale_log2 = p->scale * pa::kLog2e;
    a->debug_timeout = p->debug_timeout;
}

pa_status launch_packed(const pa::PackedAttn& a, pa_stream_t stream) {
    return cuda_status(a.dtype == PA_F32 ? pa::launch_packed_f32(a, stream) : pa::launch_packed_tc(a, stream));
}

pa_status check_pages(const pa_params* p, pa::PagesCall* c) {
    if (!p) return PA_ERR_NULL;
    if (p->num_seqs < 1 || p->num_seqs > 65535 || p->max_blocks_per_seq < 1) return PA_ERR_SHAPE;
    if (p->num_pages < 1) return PA_ERR_SHAPE;
    if (p->num_pages > pa::kMaxPoolPages) return PA_ERR_UNSUPPORTED;
    if (p->page_size != 16 && p->page_size != 32) return PA_ERR_UNSUPPORTED;
    c->num_seqs = p->num_seqs;
    c->num_pages = p->num_pages;
    c->max_blocks = p->max_blocks_per_seq;
    c->page_size = p->page_size;
    return PA_OK;
}

pa_status check_pool(const int32_t* ref, const int32_t* bt, const int32_t* cl) {
    if (!ref || !bt || !cl) return PA_ERR_NULL;
    if (!aligned(ref, 4) || !aligned(bt, 4) || !aligned(cl, 4)) return PA_ERR_ALIGN;
    return PA_OK;
}

pa_status check_pages_ws(const pa_params* p, const void* ws, size_t bytes) {
    if (!ws) return PA_ERR_NULL;
    if (bytes < pa::pages_workspace_bytes(p->num_seqs, p->num_pages)) return PA_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return PA_ERR_ALIGN;
    return PA_OK;
}

}  // namespace

PA_EXPORT pa_rows* pa_rows_init(pa_rows* r) {
    if (r) memset(r, 0, sizeof *r);
    return r;
}

PA_EXPORT pa_status pa_prompt(const pa_params* p, const pa_rows* r, const void* q, const void* k, const void* v,
                              const int32_t* cu_lens, void* out, uint32_t* dev_status, pa_stream_t stream) {
    if (!p || !r) return PA_ERR_NULL;
    pa::PackedAttn a = {};
    pa_status st = check_heads(p);
    if (st != PA_OK) return st;
    if ((st = check_rows(p, r, &a.r)) != PA_OK) return st;
    if (r->total_rows == 0) return PA_OK;
    // the kernels number their tiles of 64 or 128 (row, head) pairs in 32 bits
    const int tile = 64 / (p->num_q_heads / p->num_kv_heads);
    if (((a.r.max_rows + tile - 1) / tile) * int64_t(p->num_kv_heads) * p->num_seqs > (1 << 30))
        return PA_ERR_UNSUPPORTED;
    if (!q || !k || !v || !cu_lens || !out) return PA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_lens, 4))
        return PA_ERR_ALIGN;
    fill_heads(p, &a);
    a.r.cu_lens = cu_lens;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.dev_status = dev_status;
    a.n_ctas = share_ctas(p);
    return launch_packed(a, stream);
}

PA_EXPORT size_t pa_tree_workspace_size(const pa_params* p, const pa_rows* r) {
    pa::PackedAttn a = {};
    if (check_tree(p, r, &a) != PA_OK) return 0;
    return tree_bytes(p, a.n_ctas);
}

PA_EXPORT pa_status pa_tree(const pa_params* p, const pa_rows* r, const void* q, const void* k, const void* v,
                            const int32_t* cu_lens, const uint32_t* tree_mask, const void* k_cache,
                            const void* v_cache, const int32_t* block_tables, const int32_t* context_lens, void* out,
                            void* workspace, size_t workspace_bytes, uint32_t* dev_status, pa_stream_t stream) {
    pa::PackedAttn a = {};
    pa_status st = check_tree(p, r, &a);
    if (st != PA_OK) return st;
    if (r->total_rows == 0) return PA_OK;
    if (!q || !k || !v || !cu_lens || !tree_mask || !k_cache || !v_cache || !block_tables || !context_lens || !out ||
        !workspace)
        return PA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(cu_lens, 4) || !aligned(tree_mask, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(workspace, 256))
        return PA_ERR_ALIGN;
    if (workspace_bytes < tree_bytes(p, a.n_ctas)) return PA_ERR_WORKSPACE;
    fill_heads(p, &a);
    a.r.cu_lens = cu_lens;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.dev_status = dev_status;
    a.tree_mask = tree_mask;
    a.c.k = k_cache;
    a.c.v = v_cache;
    a.c.block_tables = block_tables;
    a.c.context_lens = context_lens;
    a.workspace = workspace;
    return launch_packed(a, stream);
}

PA_EXPORT pa_status pa_store(const pa_params* p, const pa_rows* r, const void* k, const void* v,
                             const int32_t* cu_lens, const int32_t* row_index, void* k_cache, void* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens, uint32_t* dev_status,
                             pa_stream_t stream) {
    if (!p || !r) return PA_ERR_NULL;
    pa::StoreCall c = {};
    pa_status st = check_cache(p, &c.c);
    if (st != PA_OK) return st;
    if ((st = check_rows(p, r, &c.r)) != PA_OK) return st;
    c.source_rows = r->source_rows ? r->source_rows : r->total_rows;
    if (!row_index && c.source_rows < r->total_rows) return PA_ERR_SHAPE;
    if (r->total_rows == 0) return PA_OK;
    if (!k || !v || !cu_lens || !k_cache || !v_cache || !block_tables || !context_lens) return PA_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(cu_lens, 4) ||
        !aligned(row_index, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PA_ERR_ALIGN;
    c.r.cu_lens = cu_lens;
    c.k = k;
    c.v = v;
    c.row_index = row_index;
    c.Hkv = p->num_kv_heads;
    c.D = p->head_dim;
    c.elt_bytes = elt_bytes(p->kv_dtype);
    c.c.k = k_cache;
    c.c.v = v_cache;
    c.c.block_tables = block_tables;
    c.c.context_lens = context_lens;
    c.dev_status = dev_status;
    return cuda_status(pa::launch_store(c, stream));
}

PA_EXPORT size_t pa_pages_workspace_size(const pa_params* p) {
    pa::PagesCall c = {};
    return check_pages(p, &c) == PA_OK ? pa::pages_workspace_bytes(p->num_seqs, p->num_pages) : 0;
}

PA_EXPORT pa_status pa_pages_resize(const pa_params* p, int32_t* refcounts, int32_t* block_tables,
                                    int32_t* context_lens, const int32_t* new_lens, int32_t* pairs, void* workspace,
                                    size_t workspace_bytes, uint32_t* dev_status, pa_stream_t stream) {
    pa::PagesCall c = {};
    pa_status st = check_pages(p, &c);
    if (st != PA_OK) return st;
    if ((st = check_pool(refcounts, block_tables, context_lens)) != PA_OK) return st;
    if (!new_lens || !pairs) return PA_ERR_NULL;
    if (!aligned(new_lens, 4) || !aligned(pairs, 8)) return PA_ERR_ALIGN;
    if ((st = check_pages_ws(p, workspace, workspace_bytes)) != PA_OK) return st;
    c.refcounts = refcounts;
    c.block_tables = block_tables;
    c.context_lens = context_lens;
    c.workspace = workspace;
    c.dev_status = dev_status;
    return cuda_status(pa::launch_pages_resize(c, new_lens, pairs, stream));
}

PA_EXPORT pa_status pa_pages_fork(const pa_params* p, int32_t* refcounts, int32_t* block_tables, int32_t* context_lens,
                                  const int32_t* src, const int32_t* dst, int32_t n, uint32_t* dev_status,
                                  pa_stream_t stream) {
    pa::PagesCall c = {};
    pa_status st = check_pages(p, &c);
    if (st != PA_OK) return st;
    if (n < 0) return PA_ERR_SHAPE;
    if (n == 0) return PA_OK;
    if ((st = check_pool(refcounts, block_tables, context_lens)) != PA_OK) return st;
    if (!src || !dst) return PA_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4)) return PA_ERR_ALIGN;
    c.refcounts = refcounts;
    c.block_tables = block_tables;
    c.context_lens = context_lens;
    c.dev_status = dev_status;
    return cuda_status(pa::launch_pages_fork(c, src, dst, n, stream));
}

PA_EXPORT pa_status pa_pages_compact(const pa_params* p, int32_t* refcounts, int32_t* block_tables,
                                     const int32_t* context_lens, int32_t* pairs, int32_t max_moves,
                                     int32_t* num_moves, void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                     pa_stream_t stream) {
    pa::PagesCall c = {};
    pa_status st = check_pages(p, &c);
    if (st != PA_OK) return st;
    if (max_moves < 0) return PA_ERR_SHAPE;
    if ((st = check_pool(refcounts, block_tables, context_lens)) != PA_OK) return st;
    if ((max_moves > 0 && !pairs) || !num_moves) return PA_ERR_NULL;
    if (!aligned(pairs, 8) || !aligned(num_moves, 4)) return PA_ERR_ALIGN;
    if ((st = check_pages_ws(p, workspace, workspace_bytes)) != PA_OK) return st;
    c.refcounts = refcounts;
    c.block_tables = block_tables;
    c.context_lens = const_cast<int32_t*>(context_lens);
    c.workspace = workspace;
    c.dev_status = dev_status;
    return cuda_status(pa::launch_pages_compact(c, pairs, max_moves, num_moves, stream));
}

PA_EXPORT pa_status pa_pages_copy(const pa_params* p, void* k_cache, void* v_cache, const int32_t* pairs, int32_t n,
                                  uint32_t* dev_status, pa_stream_t stream) {
    if (!p) return PA_ERR_NULL;
    pa::CacheArgs c = {};
    pa_status st = check_cache(p, &c);
    if (st != PA_OK) return st;
    if (n < 0) return PA_ERR_SHAPE;
    if (n == 0) return PA_OK;
    if (!k_cache || !v_cache || !pairs) return PA_ERR_NULL;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(pairs, 8)) return PA_ERR_ALIGN;
    c.k = k_cache;
    c.v = v_cache;
    return cuda_status(
        pa::launch_pages_copy(c, p->num_kv_heads, p->head_dim, elt_bytes(p->kv_dtype), pairs, n, dev_status, stream));
}
