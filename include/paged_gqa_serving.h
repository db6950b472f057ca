/*
 * paged_gqa_serving.h -- the serving-step entry points of libpaged_gqa.so,
 * beside the decode and chunked prefill of paged_gqa.h:
 *
 *   pa_prompt         causal attention over whole prompts, packed, no pages
 *   pa_store          packed K/V rows into the pages (a prompt's, or the
 *                     accepted drafts' by index)
 *   pa_tree           attention of a tree of drafted tokens over the paged
 *                     history and the drafts themselves
 *   pa_pages_resize   reserve, trim and free the pages of sequences, with
 *                     copy-on-write of a shared last page
 *   pa_pages_fork     let sequences share another's pages
 *   pa_pages_compact  move the live pages to the low end of the pool
 *   pa_pages_copy     copy pages of one layer's K and V
 *   pa_rotate         norms and rotation of queries and keys, and their store
 *   pa_verify         which drafts the target's distribution accepts
 *   pa_key_weights    the attention weight that each cached key has gathered
 *   pa_evict          drop the keys that gathered least
 *
 * A step of a serving loop: pa_pages_resize reserves room; pa_rotate,
 * pa_prompt and pa_store take a prompt in (once per layer; pa_rotate can
 * store the rows itself); then, per token or per drafted tree, pa_decode /
 * pa_tree, pa_verify, and pa_store of what was accepted.  A cache with a
 * budget calls pa_key_weights after the store and, when it is full, pa_evict
 * per layer and pa_pages_resize once; from then on a sequence's length is not its
 * next position, and pa_rotate has to be given positions.
 * pa_pages_resize and pa_pages_compact change only the bookkeeping, once
 * per step; the (source, destination) pairs that they report go to
 * pa_pages_copy once per layer, before anything else touches the pages.
 *
 * The conventions of paged_gqa.h hold: pointers are caller-owned device
 * memory; calls enqueue on `stream` and return; host-detectable errors
 * return before anything is launched; device-detected metadata errors never
 * form an out-of-range address and set bits in *dev_status; grids depend on
 * host arguments only, so every call can be captured and replayed with new
 * lengths and tables; results do not depend on timing.  A workspace is
 * scratch: its contents are ignored and nothing in it outlives the call, so
 * calls ordered one after the other (replays of several captured graphs
 * among them) may share one; calls that overlap may not.
 */
#ifndef PAGED_GQA_SERVING_H
#define PAGED_GQA_SERVING_H

#include "paged_gqa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits OR-ed into *dev_status, beside PA_DEV_BAD_PAGE and the others. */
#define PA_DEV_NO_PAGES 16u  /* pa_pages_resize: not enough free pages for a sequence */
#define PA_DEV_BAD_INDEX 32u /* a row index, sequence index, position, token, parent or page of a pair out of range */
#define PA_DEV_BAD_VALUE 64u /* pa_verify: a row of logits without a finite largest value, or random numbers that choose nothing */
#define PA_DEV_SHARED_PAGE 128u /* pa_evict: a page to be written has another holder */

/* Packed rows: sequence s owns rows cu_lens[s] .. cu_lens[s+1]-1 of q, k, v
 * and out; cu_lens is [num_seqs + 1] int32 on the device, ascending from a
 * value >= 0.  Rows before the first sequence's and behind the last one's
 * have no part in any result and are not written.  A sequence whose rows
 * leave [0, total_rows] or number more than max_rows or less than none is
 * skipped, its rows left as they were (PA_DEV_BAD_LEN).  Where ends descend
 * (flagged too), rows can belong to several sequences: each element of such a
 * row is one of its sequences' results or left as it was, and which may
 * depend on timing. */
typedef struct {
    int32_t total_rows;  /* rows of the packed tensors, at most 2^30; 0: nothing
                            to do                                                */
    int32_t max_rows;    /* host bound on the rows of one sequence               */
    int32_t source_rows; /* pa_store with row_index: rows of k and v; 0 means
                            total_rows                                           */
    int32_t mask_words;  /* pa_tree: 32-bit words of a mask row; 0 means
                            ceil(max_rows / 32), its least value                  */
    int64_t q_stride;    /* elements from a row of q to the next; 0: Hq * D       */
    int64_t k_stride;    /* of k, 0: Hkv * D.  Heads are D apart, so a slice of a */
    int64_t v_stride;    /* packed QKV projection passes as it is                 */
} pa_rows;

/* Zeroes *r.  Returns r. */
pa_rows *pa_rows_init(pa_rows *r);

/* ------------------------------------------------------------------ prompt
 * For each sequence, row t and q head h of kv head g = h / (Hq / Hkv):
 *   out[t,h] = sum_{j <= t} exp(scale q[t,h].k[j,g]) v[j,g] / sum_{j <= t} exp(scale q[t,h].k[j,g])
 * q [total_rows][Hq][D], k and v [total_rows][Hkv][D] with the rows' strides,
 * out [total_rows][Hq][D] contiguous in out_dtype: PA_F32, or the dtype of q.
 * Uses of p: num_seqs, num_q_heads, num_kv_heads (ratio at most 16),
 * head_dim 64 or 128, scale (> 0), q_dtype == kv_dtype, out_dtype,
 * deterministic, debug_timeout; its page fields are ignored.  num_seqs <= 65535.
 * Scores, softmax statistics and accumulators are fp32.  With 16-bit inputs
 * the probabilities enter P.V in 16 bits when out is 16 bits wide, each off by
 * half a step at most, and as a sum of two 16-bit parts when out is PA_F32: a
 * caller who wants 16-bit results to the last step takes PA_F32 and rounds.
 * A NaN or infinity in k or v reaches only the rows that attend it (and all
 * of them, a weight that underflows to zero aside).
 * A row's bits depend on its own sequence and, with 16-bit inputs, on
 * total_rows and max_rows: they choose how rows are grouped, for the device's
 * number of SMs or, with deterministic = 1, for 152.
 * q, k, v, out 16-byte aligned; strides multiples of 16 bytes. */
pa_status pa_prompt(const pa_params *p, const pa_rows *r, const void *q, const void *k,
                    const void *v, const int32_t *cu_lens, void *out, uint32_t *dev_status,
                    pa_stream_t stream);

/* -------------------------------------------------------------------- tree
 * T_s drafts of sequence s (its packed rows) over a history of
 * L_s = context_lens[s] cached tokens, 0 <= L_s <= max_blocks_per_seq *
 * page_size and at most 2^30; the history does not hold the drafts, whose K/V come packed in
 * k and v.  Row t attends every history key, and draft j < T_s where bit
 * j % 32 of word j / 32 of its mask row is set (its own bit is not implied).
 *   tree_mask: [total_rows][mask_words] 32-bit words.
 * A row that attends nothing is written as zeros.  T_s may be 0.  History
 * pages outside the pool are skipped (PA_DEV_BAD_PAGE); an L_s out of range
 * writes the sequence's rows as zeros (PA_DEV_BAD_LEN).
 * q, k, v, out, strides, dtypes, head dims, scale and precision as in
 * pa_prompt; the cache as in pa_decode, page_size 16 or 32.  max_rows <= 1024.
 * num_splits, sliding_window and decode_q_rows > 1 are PA_ERR_UNSUPPORTED.
 * The work is split over the keys into equal shares, one per SM (152 when
 * p->deterministic, the device's count otherwise), and the pieces joined in
 * a fixed order by a second kernel.
 * workspace: pa_tree_workspace_size bytes, 256-byte aligned (0: invalid). */
size_t pa_tree_workspace_size(const pa_params *p, const pa_rows *r);

pa_status pa_tree(const pa_params *p, const pa_rows *r, const void *q, const void *k, const void *v,
                  const int32_t *cu_lens, const uint32_t *tree_mask, const void *k_cache,
                  const void *v_cache, const int32_t *block_tables, const int32_t *context_lens,
                  void *out, void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                  pa_stream_t stream);

/* ------------------------------------------------------------------- store
 * Writes n_s = cu_lens[s+1] - cu_lens[s] rows of each sequence to its last
 * n_s positions, context_lens[s] - n_s .. context_lens[s] - 1 (context_lens
 * counts them), through the block table.  Destination row i (packed, as
 * cu_lens has it) comes from row i of k and v, or from row row_index[i]
 * where row_index is not NULL ([total_rows] int32: the accepted drafts).
 * Each position must be written once per call: no page belongs to two of
 * the call's sequences at the written slots (pa_pages_resize sees to that).
 * An L_s that is out of range or below n_s skips the sequence
 * (PA_DEV_BAD_LEN), a page outside the pool (PA_DEV_BAD_PAGE) or an index
 * outside [0, source_rows) (PA_DEV_BAD_INDEX) skips the row.
 * k, v: [source_rows][Hkv][D] in kv_dtype with the rows' strides. */
pa_status pa_store(const pa_params *p, const pa_rows *r, const void *k, const void *v,
                   const int32_t *cu_lens, const int32_t *row_index, void *k_cache, void *v_cache,
                   const int32_t *block_tables, const int32_t *context_lens, uint32_t *dev_status,
                   pa_stream_t stream);

/* ------------------------------------------------------------------- pages
 * The bookkeeping of a pool, all int32 on the device:
 *   refcounts    [num_pages]  block-table entries that hold the page; 0: free
 *   block_tables [num_seqs][max_blocks_per_seq]
 *   context_lens [num_seqs]   tokens of each sequence, in its first
 *                             ceil(L / page_size) table entries
 * Lists of page copies are [n][2] int32 (source, destination); a pair with a
 * negative entry means none.  No two calls on one pool may overlap.
 * Of p, the page and sequence counts are used, and by pa_pages_copy the
 * heads, head_dim, kv_dtype and strides. */

/* Bytes of the workspace that resize and compact need; 0: invalid. */
size_t pa_pages_workspace_size(const pa_params *p);

/* Takes each sequence s to new_lens[s] tokens ([num_seqs] int32; negative:
 * left alone; 0 frees it):
 *  - growing takes pages that were free when the call began, the lowest
 *    first, in the order of sequences and within one of blocks; shrinking
 *    releases pages and sets their table entries to -1;
 *  - the page that holds slot e = min(old, new), when e is inside a page and
 *    the page is shared (refcount > 1 when the call began), is replaced by
 *    a fresh one, taken before the sequence's other pages, and
 *    pairs[s] = (shared, fresh); otherwise pairs[s] = (-1, -1).  Run
 *    pa_pages_copy on pairs in every layer before the next write.  Each
 *    sharer that the call resizes gets a page of its own, so one that they
 *    all leave is free afterwards;
 *  - a sequence whose pages do not suffice, counting those that the
 *    sequences before it asked for, is left as it was (PA_DEV_NO_PAGES);
 *    one whose old or new length is out of range too (PA_DEV_BAD_LEN).
 * A released table entry outside the pool, of a page that was free when the
 * call began or of one whose refcount falls to 0 before it, is passed over
 * (PA_DEV_BAD_PAGE).  pairs: [num_seqs][2]. */
pa_status pa_pages_resize(const pa_params *p, int32_t *refcounts, int32_t *block_tables,
                          int32_t *context_lens, const int32_t *new_lens, int32_t *pairs,
                          void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                          pa_stream_t stream);

/* For each i < n: sequence dst[i], which must be empty (length 0), becomes a
 * copy of sequence src[i], sharing its pages (refcounts rise).  Skipped with
 * PA_DEV_BAD_INDEX: an index outside [0, num_seqs), a dst that is not empty
 * or that an earlier i names, a src that is some dst of the call; with
 * PA_DEV_BAD_LEN: a source length out of range.  An entry outside the pool
 * is copied as it is (PA_DEV_BAD_PAGE).  The next pa_pages_resize gives each
 * sharer that grows its own last page. */
pa_status pa_pages_fork(const pa_params *p, int32_t *refcounts, int32_t *block_tables,
                        int32_t *context_lens, const int32_t *src, const int32_t *dst, int32_t n,
                        uint32_t *dev_status, pa_stream_t stream);

/* With n live pages (refcount > 0), moves the r-th live page at or above
 * page n to the r-th free page below it, r < max_moves, and renames it in
 * every table: after it, with max_moves enough, the live pages are 0 .. n-1.
 * pairs [max_moves][2] gets the moves (the rest (-1, -1)) and *num_moves
 * (device) their number; run pa_pages_copy on pairs in every layer before
 * anything reads or writes the pages.  Tables of all sequences that use the
 * pool must be in block_tables; a context length out of range leaves its
 * table alone (PA_DEV_BAD_LEN). */
pa_status pa_pages_compact(const pa_params *p, int32_t *refcounts, int32_t *block_tables,
                           const int32_t *context_lens, int32_t *pairs, int32_t max_moves,
                           int32_t *num_moves, void *workspace, size_t workspace_bytes,
                           uint32_t *dev_status, pa_stream_t stream);

/* Copies page pairs[i][0] to page pairs[i][1] in k_cache and v_cache, all
 * slots and heads, for i < n; pairs with a negative entry are passed over,
 * others outside the pool too (PA_DEV_BAD_INDEX).  The copies run in no
 * order: a destination must not appear in another pair (the lists of
 * resize and compact never have one that does). */
pa_status pa_pages_copy(const pa_params *p, void *k_cache, void *v_cache, const int32_t *pairs,
                        int32_t n, uint32_t *dev_status, pa_stream_t stream);

/* ------------------------------------------------------------------ rotate
 * How pa_rotate turns the heads. */
typedef struct {
    int32_t rotary_dim;  /* leading dims of a head that turn, a multiple of 16, at
                            most D; 0: none (norms and store alone)               */
    int32_t interleaved; /* 0: dim i turns with i + rotary_dim / 2; 1: 2i with 2i + 1 */
    int32_t axes;        /* rows of positions, 1 to 3; 0 means 1                  */
    int32_t sections[3]; /* axes > 1: the first sections[0] pairs follow axis 0,
                            the next sections[1] axis 1, and so on; their sum is
                            rotary_dim / 2.  axes <= 1: zeros                      */
    int32_t table_rows;  /* rows of the table: positions are below it             */
    float eps;           /* of the norms                                          */
    int64_t q_out_stride, k_out_stride; /* elements from a row to the next; 0:
                            contiguous.  Heads are D apart                         */
} pa_rope;

/* Zeroes *t, eps = 1e-6.  Returns t. */
pa_rope *pa_rope_init(pa_rope *t);

/* For each packed row and head x of q and k:
 *   y = x * rsqrt(mean(x^2) + eps) * weight        (y = x where the weight is NULL)
 *   pair i < rotary_dim / 2 at position n:  c = table[n][i], w = table[n][rotary_dim / 2 + i]
 *   (y_a, y_b) -> (c y_a - w y_b, w y_a + c y_b)
 * computed in fp32 and rounded once.  q goes to q_out, k to k_out (where it is
 * not NULL) and, where k_cache is not NULL, k and the rows of v as they are
 * into the pages, to each sequence's last positions as in pa_store
 * (context_lens counts the rows).
 *   q_weight, k_weight: [D] in q_dtype, 16-byte aligned, either may be NULL
 *   table: [table_rows][rotary_dim] f32, cosines and sines of the angles, 16-byte aligned
 *   positions: [axes][total_rows] int32; NULL: the row's place in its sequence,
 *     context_lens[s] - n_s + t, on every axis.  After an eviction that is less than
 *     the tokens there have been: pass the positions, the rows are stored by
 *     context_lens all the same
 *   q_out, k_out: may be q and k themselves, with the same stride; no other overlap
 * context_lens may be NULL with positions and no cache; v, v_cache and
 * block_tables without a cache.  k_out and k_cache may not both be NULL.
 * A position outside [0, table_rows) leaves its row out everywhere
 * (PA_DEV_BAD_INDEX); lengths out of range leave a sequence out
 * (PA_DEV_BAD_LEN); a page outside the pool leaves out the store of the row
 * (PA_DEV_BAD_PAGE).  head_dim 64, 128 or 256. */
pa_status pa_rotate(const pa_params *p, const pa_rows *r, const pa_rope *t, const void *q, const void *k,
                    const void *v, const int32_t *cu_lens, const float *table, const int32_t *positions,
                    const int32_t *context_lens, const void *q_weight, const void *k_weight, void *q_out,
                    void *k_out, void *k_cache, void *v_cache, const int32_t *block_tables,
                    uint32_t *dev_status, pa_stream_t stream);

/* ------------------------------------------------------------------ verify
 * Which tokens of a drafted tree the target's distribution accepts.  The
 * packed rows of a sequence are the tokens whose logits the target has
 * computed: row 0 is the last chosen token, which is certain, the others are
 * drafts, each behind an earlier row of its sequence, its parent.
 *   logits:       [total_rows][vocab] of the target in q_dtype, r->q_stride
 *                 elements from a row to the next (0: vocab)
 *   draft_logits: the same of the distributions that the drafts were drawn from
 *                 (independently: the children of a row from its row), stride
 *                 r->k_stride; nothing is made of rows without children.  NULL:
 *                 each draft was certain to its drafter
 *   tokens, parents: [total_rows] int32; parents count within the sequence,
 *                 0 <= parents[t] < t; row 0's are not looked at
 *   temperature:  [num_seqs] f32; logits are divided by it; not above 0: greedy;
 *                 infinity: all finite logits alike
 *   uniform:      [total_rows] f32 in [0, 1), one for each draft
 *   noise:        [num_seqs][vocab] f32, independent exponential numbers above 0
 * From row 0 on, with p = softmax(target), q = softmax(draft) of the row (q
 * the certain token itself without draft_logits), its children are tried in
 * ascending order: child c is accepted when p(c) > 0 and uniform q(c) < p(c),
 * and the walk goes on from it; else p becomes max(p - q, 0), normalised
 * (left as it is where nothing remains).  Where no child is accepted, the next
 * token is the one with the largest p(i) / noise(i), ties to the lowest: the
 * tokens then follow the target's distribution.  Greedy: a child is accepted
 * when it is the target's largest logit, the next token is that one, ties to
 * the lowest; nothing is made of the random numbers and draft_logits.
 *   accepted:    [total_rows] int32: the packed rows of the accepted tokens, row
 *                0 of each sequence among them, sequence after sequence, then -1
 *   accepted_cu: [num_seqs + 1] int32: where each sequence's begin.  The two are
 *                the row_index and cu_lens of pa_store
 *   next_tokens: [num_seqs] int32
 *   new_lens:    [num_seqs] int32, context_lens[s] plus the accepted rows, for
 *                pa_pages_resize; both may be NULL
 * A sequence without rows, or with lengths out of range (PA_DEV_BAD_LEN),
 * accepts nothing, its next token is -1.  A draft whose token or parent is out
 * of range is passed over (PA_DEV_BAD_INDEX).  A visited row without a finite
 * largest logit (a NaN or +infinity, all -infinity) ends the walk with next
 * token -1 (PA_DEV_BAD_VALUE), as do random numbers that choose none.
 * -infinity in other logits is a probability of zero.
 * Uses of p: num_seqs, q_dtype, debug_timeout (1: the first exchange of a
 * sequence's first CTA gives up at once, testing).  After PA_DEV_TIMEOUT what the
 * call writes is void.  vocab from 1 to 2^28, max_rows <= 1024; logits
 * and noise aligned to their elements.  Where total_rows is 0, what has an entry
 * or more a row, temperature and noise may be NULL. */
pa_status pa_verify(const pa_params *p, const pa_rows *r, int32_t vocab, const void *logits,
                    const void *draft_logits, const int32_t *tokens, const int32_t *parents,
                    const int32_t *cu_lens, const float *temperature, const float *uniform,
                    const float *noise, const int32_t *context_lens, int32_t *accepted,
                    int32_t *accepted_cu, int32_t *next_tokens, int32_t *new_lens, uint32_t *dev_status,
                    pa_stream_t stream);

/* ------------------------------------------------------------- key weights
 * What each cached key gathers of its sequence's rows' attention:
 *   weights[s][g][j] = decay weights[s][g][j]
 *     + sum over rows t and q heads h of kv head g of
 *       exp(scale q[t,h].k_j) / sum_{i <= e_t} exp(scale q[t,h].k_i)   for j <= e_t
 * with row t of T_s seeing keys 0 ..= e_t = context_lens[s] - T_s + t, as in
 * pa_prefill_chunk (T_s = 1: a decode step); the rows' own K is in the pages.
 *   weights: [num_seqs][num_kv_heads][max_blocks_per_seq * page_size] f32.  What
 *     stood at the last T_s positions is not read, nor anything where decay is 0;
 *     places from context_lens[s] on are left as they were
 * decay in [0, 1].  A sequence without rows is left as it was.  Keys in pages
 * outside the pool take no part (PA_DEV_BAD_PAGE), theirs is decay alone.  A
 * score of -infinity weighs nothing; a NaN or +infinity makes what its row
 * adds NaN.  Finite scores may have any size.  Sums, largest scores and weights are
 * fp32; with 16-bit types and max_rows G above 32, a row's largest score below 128 (in
 * base 2) and the logarithm of its sum are one fp32 number, whose rounding (2^-18 at
 * most) is in that row's weights.
 * Uses of p as in pa_tree (head_dim 64 or 128; out_dtype is not used; no
 * windows, splits or decode_q_rows); max_context_len is a bound on
 * every context_lens[s] (0: what a table holds): longer ones are
 * PA_DEV_BAD_LEN, their weights left as they were.  deterministic: the work is
 * shared out as on 152 SMs.  debug_timeout bears on the tensor-core kernel alone;
 * after PA_DEV_TIMEOUT the weights are void.
 * (max_rows G / 64 + 8) (longest context / 128 + 8) is at most 2^30,
 * num_seqs num_kv_heads (longest context + 1) at most 2^40
 * (PA_ERR_UNSUPPORTED).
 * workspace: pa_key_weights_workspace_size bytes, 256-byte aligned (0: invalid).
 * max_rows G up to 32 (decoding): the scores, num_seqs x num_kv_heads x
 * longest context x max_rows G floats (max_rows G rounded up to even), and a pair of
 * floats for each of these columns and each 64 keys of the longest context and two
 * more (3 % of the scores in long contexts, a quarter at 16 keys), so a tight
 * max_context_len pays: it counts for every sequence.  Beyond: 8 bytes for each row
 * and q head, and 1 MB at most.
 * Which of the two a call is goes by max_rows for the whole call: a few rows more of
 * one sequence cost the single tokens beside it twice their time, in a call of their
 * own they would not.
 * It carries nothing from one call to the next. */
size_t pa_key_weights_workspace_size(const pa_params *p, const pa_rows *r);

pa_status pa_key_weights(const pa_params *p, const pa_rows *r, const void *q, const int32_t *cu_lens,
                         const void *k_cache, const int32_t *block_tables, const int32_t *context_lens,
                         float decay, float *weights, void *workspace, size_t workspace_bytes,
                         uint32_t *dev_status, pa_stream_t stream);

/* ------------------------------------------------------------------- evict
 * Takes each sequence s with 0 <= keep_lens[s] < context_lens[s] down to
 * n = keep_lens[s] keys, each kv head for itself: its last r = min(recent, n)
 * keys stay, its first f = min(first, n - r), and of the others the n - r - f
 * with the largest weights (ties to the lowest position; a NaN counts as
 * -infinity).  They keep their order and move together to slots 0 .. n-1.
 *   kept:        [num_seqs][num_kv_heads][max_blocks_per_seq * page_size] int32:
 *                entry j < n is the slot that key j came from
 *   weights_out: as weights; entry j < n is key j's weight
 *   new_lens:    [num_seqs] int32: n, or -1 where nothing was evicted
 * Sequences with keep_lens[s] negative or not below context_lens[s] keep all:
 * kept and weights_out are filled as for n = context_lens[s].  Entries from n
 * on are left as they were.  weights_out must not overlap weights, nor new_lens
 * keep_lens or context_lens (PA_ERR_SHAPE).
 * context_lens and the tables stay as they are: after the last layer,
 * pa_pages_resize with new_lens trims every sequence and frees its pages.
 * Kept keys have the positions that they were turned at; the caller counts on from
 * the tokens there have been (positions of pa_rotate).
 * refcounts ([num_pages], may be NULL): a sequence of which a page from slot f
 * to slot n - 1 has more than one holder is not evicted (PA_DEV_SHARED_PAGE).
 * Without them no such page may belong to two sequences; nor may a page stand
 * twice in one table, with or without them.  Keys whose old or new
 * page is outside the pool do not move (PA_DEV_BAD_PAGE); a length out of range
 * leaves the sequence out, new_lens -1 (PA_DEV_BAD_LEN).
 * Uses of p: num_seqs, num_kv_heads, head_dim (64, 128, 256), kv_dtype and the
 * pages.  max_blocks_per_seq * page_size is at most 2^22, num_seqs * num_kv_heads
 * at most 2^23 (PA_ERR_UNSUPPORTED). */
pa_status pa_evict(const pa_params *p, void *k_cache, void *v_cache, const int32_t *block_tables,
                   const int32_t *context_lens, const int32_t *refcounts, const float *weights,
                   const int32_t *keep_lens, int32_t first, int32_t recent, float *weights_out,
                   int32_t *kept, int32_t *new_lens, uint32_t *dev_status, pa_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* PAGED_GQA_SERVING_H */
