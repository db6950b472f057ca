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
 *
 * A step of a serving loop: pa_pages_resize reserves room; pa_prompt and
 * pa_store take a prompt in (pa_store once per layer); then, per token or
 * per drafted tree, pa_decode / pa_tree, and pa_store of what was accepted.
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
#define PA_DEV_BAD_INDEX 32u /* a row index, sequence index or page of a pair out of range */

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

#ifdef __cplusplus
}
#endif
#endif /* PAGED_GQA_SERVING_H */
