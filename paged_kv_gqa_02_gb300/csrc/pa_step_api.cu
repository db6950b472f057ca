// pa_step_api.cu -- the extern "C" entry points of paged_gqa_serving.h around
// the step's attention (rotation, draft verification, key weights, eviction):
// host-side validation (before any device access) and dispatch.  No entry point
// allocates memory.
#include <string.h>

#include "pa_checks.h"

#define PA_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr int kMaxVocab = 1 << 28;        // tokens of a vocabulary: indices with a tile stay in 32 bits
constexpr int64_t kMaxEvictUnits = 1 << 23;  // sequences times kv heads of an eviction: its grids stay in 31 bits
constexpr int64_t kMaxWeights = int64_t(1) << 40;  // of a call: their scores' bytes stay in 64 bits

// Whether n bytes at a and n at b have some in common.
bool overlap(const void* a, const void* b, int64_t n) {
    const int64_t d = static_cast<const char*>(a) - static_cast<const char*>(b);
    return d < n && -d < n;
}

// What pa_key_weights takes of the parameters.
pa_status check_key_weights(const pa_params* p, const pa_rows* r, pa::KeyWeightsCall* c) {
    if (!p || !r) return PA_ERR_NULL;
    pa_params heads = *p;
    heads.out_dtype = PA_F32;  // not used
    pa_status st = check_heads(&heads);
    if (st != PA_OK) return st;
    if ((st = check_cache(p, &c->c)) != PA_OK) return st;
    if ((st = check_rows(p, r, &c->r)) != PA_OK) return st;
    if (p->deterministic != 0 && p->deterministic != 1) return PA_ERR_SHAPE;
    if (p->num_splits != 0 || p->sliding_window != 0 || p->decode_q_rows > 1) return PA_ERR_UNSUPPORTED;
    if (p->max_context_len < 0) return PA_ERR_SHAPE;
    int64_t len = int64_t(p->max_blocks_per_seq) * p->page_size;
    if (len > kMaxHistory) len = kMaxHistory;
    if (p->max_context_len && p->max_context_len < len) len = p->max_context_len;
    c->max_len = int(len);
    // products of a kv head are numbered in tiles of at least 65 x 128, in 32 bits
    if ((int64_t(c->r.max_rows) * (p->num_q_heads / p->num_kv_heads) / 64 + 8) * (len / 128 + 8) > (1 << 30))
        return PA_ERR_UNSUPPORTED;
    if (int64_t(p->num_seqs) * p->num_kv_heads > kMaxWeights / (len + 1)) return PA_ERR_UNSUPPORTED;
    c->dtype = p->q_dtype;
    c->Hq = p->num_q_heads;
    c->Hkv = p->num_kv_heads;
    c->D = p->head_dim;
    c->n_ctas = share_ctas(p);
    c->scale_log2 = p->scale * pa::kLog2e;
    c->debug_timeout = p->debug_timeout;
    return PA_OK;
}

}  // namespace

PA_EXPORT pa_rope* pa_rope_init(pa_rope* t) {
    if (t) {
        memset(t, 0, sizeof *t);
        t->eps = 1e-6f;
    }
    return t;
}

PA_EXPORT pa_status pa_rotate(const pa_params* p, const pa_rows* r, const pa_rope* t, const void* q, const void* k,
                              const void* v, const int32_t* cu_lens, const float* table, const int32_t* positions,
                              const int32_t* context_lens, const void* q_weight, const void* k_weight, void* q_out,
                              void* k_out, void* k_cache, void* v_cache, const int32_t* block_tables,
                              uint32_t* dev_status, pa_stream_t stream) {
    if (!p || !r || !t) return PA_ERR_NULL;
    pa::RotateCall c = {};
    if (p->num_seqs < 1 || p->num_seqs > 65535 || p->num_q_heads < 1 || p->num_kv_heads < 1 ||
        p->num_q_heads > 65535 || p->num_kv_heads > 65535)
        return PA_ERR_SHAPE;
    if (!known_dtype(p->q_dtype) || !known_dtype(p->kv_dtype)) return PA_ERR_DTYPE;
    if (p->q_dtype != p->kv_dtype) return PA_ERR_UNSUPPORTED;
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return PA_ERR_UNSUPPORTED;
    pa_status st;
    if (k_cache && (st = check_cache(p, &c.c)) != PA_OK) return st;
    if ((st = check_rows(p, r, &c.r)) != PA_OK) return st;
    c.t = *t;
    if (t->rotary_dim < 0 || t->rotary_dim > p->head_dim || t->rotary_dim % 16) return PA_ERR_SHAPE;
    if (t->interleaved != 0 && t->interleaved != 1) return PA_ERR_SHAPE;
    if (t->axes < 0 || t->axes > 3 || !(t->eps >= 0.f) || !isfinite(t->eps)) return PA_ERR_SHAPE;
    if (t->rotary_dim && t->table_rows < 1) return PA_ERR_SHAPE;
    if (t->axes == 0) c.t.axes = 1;
    int64_t pairs = 0;
    for (int i = 0; i < 3; ++i) {
        if (t->sections[i] < 0 || (t->sections[i] && i >= t->axes)) return PA_ERR_SHAPE;
        pairs += t->sections[i];
    }
    if (c.t.axes > 1 ? pairs != t->rotary_dim / 2 : pairs != 0) return PA_ERR_SHAPE;
    const int eb = elt_bytes(p->q_dtype);
    const int64_t nq = int64_t(p->head_dim) * p->num_q_heads, nk = int64_t(p->head_dim) * p->num_kv_heads;
    if (!t->q_out_stride) c.t.q_out_stride = nq;
    if (!t->k_out_stride) c.t.k_out_stride = nk;
    if (c.t.q_out_stride < nq || c.t.k_out_stride < nk) return PA_ERR_SHAPE;
    if ((c.t.q_out_stride * eb) % 16 || (c.t.k_out_stride * eb) % 16) return PA_ERR_ALIGN;
    if (r->total_rows == 0) return PA_OK;
    if (!q || !k || !cu_lens || !q_out || (!k_out && !k_cache)) return PA_ERR_NULL;
    if (t->rotary_dim && !table) return PA_ERR_NULL;
    if (k_cache ? !v || !v_cache || !block_tables || !context_lens : !positions && !context_lens) return PA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(table, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(cu_lens, 4) || !aligned(positions, 4) || !aligned(context_lens, 4) ||
        !aligned(block_tables, 4))
        return PA_ERR_ALIGN;
    // rows that are written over their input have to lie as it does
    if ((q_out == q && c.t.q_out_stride != c.r.q_stride) || (k_out && k_out == k && c.t.k_out_stride != c.r.k_stride))
        return PA_ERR_SHAPE;
    c.r.cu_lens = cu_lens;
    c.q = q;
    c.k = k;
    c.v = v;
    c.q_weight = q_weight;
    c.k_weight = k_weight;
    c.q_out = q_out;
    c.k_out = k_out;
    c.table = table;
    c.positions = positions;
    c.dtype = p->q_dtype;
    c.Hq = p->num_q_heads;
    c.Hkv = p->num_kv_heads;
    c.D = p->head_dim;
    c.c.k = k_cache;
    c.c.v = v_cache;
    c.c.block_tables = block_tables;
    c.c.context_lens = context_lens;
    c.dev_status = dev_status;
    return cuda_status(pa::launch_rotate(c, stream));
}

PA_EXPORT pa_status pa_verify(const pa_params* p, const pa_rows* r, int32_t vocab, const void* logits,
                              const void* draft_logits, const int32_t* tokens, const int32_t* parents,
                              const int32_t* cu_lens, const float* temperature, const float* uniform,
                              const float* noise, const int32_t* context_lens, int32_t* accepted,
                              int32_t* accepted_cu, int32_t* next_tokens, int32_t* new_lens, uint32_t* dev_status,
                              pa_stream_t stream) {
    if (!p || !r) return PA_ERR_NULL;
    pa::VerifyCall c = {};
    if (p->num_seqs < 1 || p->num_seqs > 65535) return PA_ERR_SHAPE;
    if (!known_dtype(p->q_dtype)) return PA_ERR_DTYPE;
    if (r->total_rows < 0 || r->max_rows < 0 || (r->total_rows > 0 && r->max_rows < 1)) return PA_ERR_SHAPE;
    if (vocab < 1) return PA_ERR_SHAPE;
    c.max_rows = r->max_rows < r->total_rows ? r->max_rows : r->total_rows;
    if (r->total_rows > kMaxRows || c.max_rows > kMaxTreeRows || vocab > kMaxVocab) return PA_ERR_UNSUPPORTED;
    c.logits_stride = r->q_stride ? r->q_stride : vocab;
    c.draft_stride = r->k_stride ? r->k_stride : vocab;
    if (c.logits_stride < vocab || c.draft_stride < vocab) return PA_ERR_SHAPE;
    if (!cu_lens || !accepted_cu || !next_tokens || !context_lens != !new_lens) return PA_ERR_NULL;
    if (r->total_rows > 0 && (!logits || !tokens || !parents || !temperature || !uniform || !noise || !accepted))
        return PA_ERR_NULL;
    const unsigned eb = elt_bytes(p->q_dtype);
    if (!aligned(logits, eb) || !aligned(draft_logits, eb) || !aligned(tokens, 4) || !aligned(parents, 4) ||
        !aligned(cu_lens, 4) || !aligned(temperature, 4) || !aligned(uniform, 4) || !aligned(noise, 4) ||
        !aligned(context_lens, 4) || !aligned(accepted, 4) || !aligned(accepted_cu, 4) || !aligned(next_tokens, 4) ||
        !aligned(new_lens, 4))
        return PA_ERR_ALIGN;
    c.cu_lens = cu_lens;
    c.logits = logits;
    c.draft = draft_logits;
    c.tokens = tokens;
    c.parents = parents;
    c.temperature = temperature;
    c.uniform = uniform;
    c.noise = noise;
    c.context_lens = context_lens;
    c.accepted = accepted;
    c.accepted_cu = accepted_cu;
    c.next_tokens = next_tokens;
    c.new_lens = new_lens;
    c.num_seqs = p->num_seqs;
    c.total_rows = r->total_rows;
    c.vocab = vocab;
    c.dtype = p->q_dtype;
    c.dev_status = dev_status;
    c.debug_timeout = p->debug_timeout == 1;
    return cuda_status(pa::launch_verify(c, stream));
}

PA_EXPORT size_t pa_key_weights_workspace_size(const pa_params* p, const pa_rows* r) {
    pa::KeyWeightsCall c = {};
    return check_key_weights(p, r, &c) == PA_OK ? pa::key_weights_workspace_bytes(c) : 0;
}

PA_EXPORT pa_status pa_key_weights(const pa_params* p, const pa_rows* r, const void* q, const int32_t* cu_lens,
                                   const void* k_cache, const int32_t* block_tables, const int32_t* context_lens,
                                   float decay, float* weights, void* workspace, size_t workspace_bytes,
                                   uint32_t* dev_status, pa_stream_t stream) {
    pa::KeyWeightsCall c = {};
    const pa_status st = check_key_weights(p, r, &c);
    if (st != PA_OK) return st;
    if (!(decay >= 0.f && decay <= 1.f)) return PA_ERR_SHAPE;
    if (r->total_rows == 0) return PA_OK;
    if (!q || !cu_lens || !k_cache || !block_tables || !context_lens || !weights || !workspace) return PA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(weights, 16) || !aligned(cu_lens, 4) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(workspace, 256))
        return PA_ERR_ALIGN;
    if (workspace_bytes < pa::key_weights_workspace_bytes(c)) return PA_ERR_WORKSPACE;
    c.r.cu_lens = cu_lens;
    c.q = q;
    c.c.k = k_cache;
    c.c.block_tables = block_tables;
    c.c.context_lens = context_lens;
    c.weights = weights;
    c.decay = decay;
    c.workspace = workspace;
    c.dev_status = dev_status;
    return cuda_status(pa::launch_key_weights(c, stream));
}

PA_EXPORT pa_status pa_evict(const pa_params* p, void* k_cache, void* v_cache, const int32_t* block_tables,
                             const int32_t* context_lens, const int32_t* refcounts, const float* weights,
                             const int32_t* keep_lens, int32_t first, int32_t recent, float* weights_out,
                             int32_t* kept, int32_t* new_lens, uint32_t* dev_status, pa_stream_t stream) {
    if (!p) return PA_ERR_NULL;
    pa::EvictCall c = {};
    const pa_status st = check_cache(p, &c.c);
    if (st != PA_OK) return st;
    if (first < 0 || recent < 0) return PA_ERR_SHAPE;
    if (int64_t(p->max_blocks_per_seq) * p->page_size > pa::kMaxEvictSlots ||
        int64_t(p->num_seqs) * p->num_kv_heads > kMaxEvictUnits)
        return PA_ERR_UNSUPPORTED;
    if (!k_cache || !v_cache || !block_tables || !context_lens || !weights || !keep_lens || !weights_out || !kept ||
        !new_lens)
        return PA_ERR_NULL;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(refcounts, 4) || !aligned(weights, 16) || !aligned(keep_lens, 4) || !aligned(weights_out, 16) ||
        !aligned(kept, 16) || !aligned(new_lens, 4))
        return PA_ERR_ALIGN;
    const int64_t lens = int64_t(p->num_seqs) * 4;
    const int64_t table = lens * p->num_kv_heads * p->max_blocks_per_seq * p->page_size;
    // new_lens of a sequence is written while CTAs of its other heads may still read its lengths
    if (overlap(weights_out, weights, table) || overlap(new_lens, keep_lens, lens) || overlap(new_lens, context_lens, lens))
        return PA_ERR_SHAPE;
    c.c.k = k_cache;
    c.c.v = v_cache;
    c.c.block_tables = block_tables;
    c.c.context_lens = context_lens;
    c.refcounts = refcounts;
    c.weights = weights;
    c.keep_lens = keep_lens;
    c.weights_out = weights_out;
    c.kept = kept;
    c.new_lens = new_lens;
    c.num_seqs = p->num_seqs;
    c.Hkv = p->num_kv_heads;
    c.D = p->head_dim;
    c.elt_bytes = elt_bytes(p->kv_dtype);
    c.first = first;
    c.recent = recent;
    c.dev_status = dev_status;
    return cuda_status(pa::launch_evict(c, stream));
}
