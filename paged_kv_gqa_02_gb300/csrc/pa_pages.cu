// pa_pages.cu -- the operations on the pages of a pool and the K/V store.
//
// Bookkeeping (resize, compact) needs "the k-th free page" for many k at
// once.  No free list is kept: a refcount of 0 is what makes a page free, so
// the answer depends on the refcounts alone and the same call always hands
// out the same pages.  A first kernel cuts the refcounts into chunks of 2,048
// and leaves each chunk's free pages, ascending, and their number; the second
// kernel's CTAs sum the chunk counts (a few dozen in a usual pool) and find
// their pages by binary search.  The second kernel is launched with
// programmatic dependent launch, so that the pair costs about one launch.
//
// The copies are bound by HBM: 16-byte loads, eight in flight per thread.
#include "pa_ptx.cuh"
#include "pa_serving.h"

namespace pa {

namespace {

constexpr int kChunk = 2048;                        // pages a CTA of the scan looks through
constexpr int kScanThr = 256;
constexpr int kWarps = kScanThr / 32;

// Workspace: inclusive needs of each sequence within its block of 256 and
// block totals (64 bits: absurd lengths must not wrap), then in 32 bits chunk
// counts, chunk lists (free pages), and the page map of compact or, of resize,
// a bit for each page that was free when the call began.
struct PagesWs {
    int64_t* need;
    int64_t* block_need;
    int32_t* count;
    int32_t* list;
    int32_t* map;
    uint32_t* was_free;  // in the map's place
};
__host__ __device__ inline int n_chunks(int pages) { return (pages + kChunk - 1) / kChunk; }
__host__ __device__ inline int n_blocks(int seqs) { return (seqs + kScanThr - 1) / kScanThr; }
__host__ __device__ inline PagesWs ws_of(void* ws, int seqs, int pages) {
    PagesWs w;
    w.need = static_cast<int64_t*>(ws);
    w.block_need = w.need + seqs;
    w.count = reinterpret_cast<int32_t*>(w.block_need + n_blocks(seqs));
    w.list = w.count + n_chunks(pages);
    w.map = w.list + int64_t(n_chunks(pages)) * kChunk;
    w.was_free = reinterpret_cast<uint32_t*>(w.map);
    return w;
}

// A sequence's part in a resize: its pages before and after, and whether the
// page of its last kept slot has to be replaced.
struct Plan {
    int had, has, edge_block;
    bool asked, bad, copy;
};

__device__ inline Plan plan_of(const PagesCall& c, const int32_t* new_lens, int s) {
    Plan p = {0, 0, 0, false, false, false};
    const int L = c.context_lens[s], N = new_lens[s];
    const int64_t cap = int64_t(c.max_blocks) * c.page_size;
    p.bad = L < 0 || L > cap || N > cap;
    p.asked = !p.bad && N >= 0;
    if (!p.asked) return p;
    const int P = c.page_size, edge = min(L, N);
    p.had = L / P + (L % P != 0);
    p.has = N / P + (N % P != 0);
    p.edge_block = edge / P;
    if (edge % P) {
        const int pg = c.block_tables[int64_t(s) * c.max_blocks + p.edge_block];
        p.copy = pg >= 0 && pg < c.num_pages && c.refcounts[pg] > 1;
    }
    return p;
}

constexpr int64_t kCopyBit = int64_t(1) << 62;  // in a need word: the first page replaces a shared one

// Inclusive sum over the CTA's threads (kScanThr of them); the warps' sums stay in warp_sums.
template <typename N> __device__ inline N block_scan(N v, N* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += warp_sums[w];
    return v;
}

// CTAs [0, n_chunks): the free pages of a chunk.  CTAs behind them (resize
// only): what 256 sequences each ask for.
__global__ void __launch_bounds__(kScanThr) pages_scan(const PagesCall c, const int32_t* new_lens) {
    __shared__ int sums[kWarps];
    __shared__ int64_t sums64[kWarps];
    pdl_wait_primary();
    pdl_launch_dependents();  // after the wait: the next kernel may not overtake the one before this
    const PagesWs w = ws_of(c.workspace, c.num_seqs, c.num_pages);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nc = n_chunks(c.num_pages);
    if (int(blockIdx.x) < nc) {
        constexpr int kPer = kChunk / kScanThr;
        const int base = int(blockIdx.x) * kChunk + warp * (32 * kPer);
        bool free_[kPer];
        int n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int page = base + 32 * i + lane;
            free_[i] = page < c.num_pages && c.refcounts[page] == 0;
        }
        unsigned m[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            m[i] = __ballot_sync(0xffffffffu, free_[i]);
            n += __popc(m[i]);
        }
        if (lane == 0) sums[warp] = n;
        __syncthreads();
        int at = 0, all = 0;
        for (int x = 0; x < kWarps; ++x) {
            if (x < warp) at += sums[x];
            all += sums[x];
        }
        int32_t* list = w.list + int64_t(blockIdx.x) * kChunk;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (free_[i]) list[at + __popc(m[i] & ((1u << lane) - 1u))] = base + 32 * i + lane;
            if (new_lens && lane == 0 && base + 32 * i < c.num_pages) w.was_free[base / 32 + i] = m[i];
            at += __popc(m[i]);
        }
        if (tid == 0) w.count[blockIdx.x] = all;
        return;
    }
    const int blk = int(blockIdx.x) - nc;
    const int s = blk * kScanThr + tid;
    int need = 0;
    Plan p = {0, 0, 0, false, false, false};
    if (s < c.num_seqs) {
        p = plan_of(c, new_lens, s);
        if (p.bad) flag(c.dev_status, PA_DEV_BAD_LEN);
        need = max(0, p.has - p.had) + (p.copy ? 1 : 0);
    }
    const int64_t upto = block_scan<int64_t>(need, sums64);
    if (s < c.num_seqs) w.need[s] = upto | (p.copy ? kCopyBit : 0);
    if (tid == kScanThr - 1) w.block_need[blk] = upto;
}

// Exclusive prefix sums of n counts into pre (shared memory); returns the total.
__device__ inline int prefix_counts(const int32_t* counts, int n, int* pre, int* sums) {
    int carry = 0;
    for (int b = 0; b < n; b += kScanThr) {
        const int i = b + int(threadIdx.x);
        const int v = i < n ? counts[i] : 0;
        const int upto = block_scan(v, sums);
        if (i < n) pre[i] = carry + upto - v;
        int tile = 0;  // of this tile, from the warps' sums
        for (int w = 0; w < kWarps; ++w) tile += sums[w];
        carry += tile;
    }
    __syncthreads();
    return carry;
}

// The k-th free page (k below their number).
__device__ inline int free_page(const PagesWs& w, const int* pre, int n, int k) {
    int lo = 0, hi = n - 1;  // the last chunk whose prefix is <= k holds it (empty chunks share the next one's prefix)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= k)
            lo = mid;
        else
            hi = mid - 1;
    }
    return w.list[int64_t(lo) * kChunk + (k - pre[lo])];
}

// Gives back one hold on a table entry.  A page that was free when the call
// began may be another sequence's by now: no hold on it is given back.
__device__ inline void release(const PagesCall& c, const PagesWs& w, int pg) {
    if (pg < 0 || pg >= c.num_pages || ((w.was_free[pg >> 5] >> (pg & 31)) & 1u)) {
        flag(c.dev_status, PA_DEV_BAD_PAGE);
    } else if (atomicSub(c.refcounts + pg, 1) <= 0) {
        atomicAdd(c.refcounts + pg, 1);
        flag(c.dev_status, PA_DEV_BAD_PAGE);
    }
}

// One CTA per sequence.  Refcounts are changed only here, after the scan has
// read them all; integer atomics, whose order does not matter.
__global__ void __launch_bounds__(kScanThr) pages_resize(const PagesCall c, const int32_t* new_lens, int32_t* pairs) {
    extern __shared__ int pre[];
    __shared__ int sums[kWarps];
    __shared__ int64_t sums64[kWarps];
    pdl_wait_primary();
    const PagesWs w = ws_of(c.workspace, c.num_seqs, c.num_pages);
    const int s = blockIdx.x, tid = threadIdx.x, nc = n_chunks(c.num_pages);
    const int L = c.context_lens[s], N = new_lens[s], P = c.page_size;
    const int64_t cap = int64_t(c.max_blocks) * P;
    int32_t* pair = pairs + 2 * int64_t(s);
    __syncthreads();  // every thread has read L, which the first one writes
    if (L < 0 || L > cap || N > cap || N < 0) {
        if (tid < 2) pair[tid] = -1;
        return;
    }
    const int had = L / P + (L % P != 0), has = N / P + (N % P != 0);
    const bool copy = w.need[s] & kCopyBit;
    const int need = max(0, has - had) + (copy ? 1 : 0);
    // the free pages before this sequence's: those that the sequences before it asked for
    int first = 0;
    if (need) {
        int64_t v = 0;
        for (int i = tid; i < s / kScanThr; i += kScanThr) v += w.block_need[i];
        block_scan<int64_t>(v, sums64);
        int64_t before = (w.need[s] & ~kCopyBit) - need;
        for (int x = 0; x < kWarps; ++x) before += sums64[x];
        const int have = prefix_counts(w.count, nc, pre, sums);
        if (before + need > have) {
            if (tid == 0) flag(c.dev_status, PA_DEV_NO_PAGES);
            if (tid < 2) pair[tid] = -1;
            return;
        }
        first = int(before);
    }
    int32_t* row = c.block_tables + int64_t(s) * c.max_blocks;
    if (tid == 0) {
        int from = -1, to = -1;
        if (copy) {
            const int b = min(L, N) / P;
            from = row[b];
            to = free_page(w, pre, nc, first);
            row[b] = to;
            atomicAdd(c.refcounts + to, 1);
            release(c, w, from);  // shared by more entries than it counts: flagged
        }
        pair[0] = from;
        pair[1] = to;
        c.context_lens[s] = N;
    }
    for (int b = had + tid; b < has; b += kScanThr) {
        const int pg = free_page(w, pre, nc, first + (copy ? 1 : 0) + b - had);
        row[b] = pg;
        atomicAdd(c.refcounts + pg, 1);
    }
    for (int b = has + tid; b < had; b += kScanThr) {
        release(c, w, row[b]);
        row[b] = -1;
    }
}

// One CTA per (source, destination).
__global__ void __launch_bounds__(kScanThr)
    pages_fork(const PagesCall c, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n) {
    pdl_wait_primary();
    const int i = blockIdx.x, tid = threadIdx.x;
    const int from = src[i], to = dst[i];
    bool bad = from < 0 || from >= c.num_seqs || to < 0 || to >= c.num_seqs;
    // Lengths are read only where no CTA of this call writes them: `to` before
    // this CTA writes it, `from` when it is no destination.
    for (int j = tid; j < n; j += kScanThr) bad |= dst[j] == from || (j < i && dst[j] == to);
    if (__syncthreads_or(bad)) {
        if (tid == 0) flag(c.dev_status, PA_DEV_BAD_INDEX);
        return;
    }
    const int L = c.context_lens[from], was = c.context_lens[to];
    const bool bad_len = L < 0 || L > int64_t(c.max_blocks) * c.page_size;
    __syncthreads();  // every thread has read `was`
    if (was != 0 || bad_len) {
        if (tid == 0) flag(c.dev_status, was != 0 ? PA_DEV_BAD_INDEX : PA_DEV_BAD_LEN);
        return;
    }
    const int used = L / c.page_size + (L % c.page_size != 0);
    const int32_t* a = c.block_tables + int64_t(from) * c.max_blocks;
    int32_t* b = c.block_tables + int64_t(to) * c.max_blocks;
    for (int k = tid; k < used; k += kScanThr) {
        const int pg = a[k];
        b[k] = pg;
        if (pg >= 0 && pg < c.num_pages)
            atomicAdd(c.refcounts + pg, 1);
        else
            flag(c.dev_status, PA_DEV_BAD_PAGE);
    }
    if (tid == 0) c.context_lens[to] = L;
}

// After the scan: pages at or above the number of live ones move down.  One
// CTA per chunk; a CTA writes the refcounts of its own high pages and of
// their holes, all below the live count, where no CTA reads any.
__global__ void __launch_bounds__(kScanThr)
    pages_compact(const PagesCall c, int32_t* pairs, int max_moves, int32_t* num_moves) {
    extern __shared__ int pre[];
    __shared__ int sums[kWarps];
    __shared__ int low_holes;
    pdl_wait_primary();
    pdl_launch_dependents();
    const PagesWs w = ws_of(c.workspace, c.num_seqs, c.num_pages);
    const int tid = threadIdx.x, nc = n_chunks(c.num_pages);
    const int n_free = prefix_counts(w.count, nc, pre, sums);
    const int live = c.num_pages - n_free;
    if (tid == 0) {  // free pages below `live`: by the prefix, then within its chunk
        int k = n_free;
        if (live < c.num_pages) {
            const int ch = live / kChunk;
            const int32_t* list = w.list + int64_t(ch) * kChunk;
            int lo = 0, hi = w.count[ch];
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (list[mid] < live)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            k = pre[ch] + lo;
        }
        low_holes = k;
    }
    __syncthreads();
    const int moves = low_holes;  // holes below = live pages above
    const int done = min(moves, max_moves);
    if (blockIdx.x == 0 && tid == 0) *num_moves = done;
    for (int i = done + int(blockIdx.x) * kScanThr + tid; i < max_moves; i += int(gridDim.x) * kScanThr)
        reinterpret_cast<int2*>(pairs)[i] = make_int2(-1, -1);
    const int page0 = int(blockIdx.x) * kChunk;
    if (page0 + kChunk <= live) return;
    const int32_t* list = w.list + int64_t(blockIdx.x) * kChunk;
    const int n_list = w.count[blockIdx.x];
    for (int i = tid; i < kChunk; i += kScanThr) {
        const int page = page0 + i;
        if (page < live || page >= c.num_pages) continue;
        int to = page;
        const int ref = c.refcounts[page];
        if (ref != 0) {
            int lo = 0, hi = n_list;  // free pages of the chunk before this one
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (list[mid] < page)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            const int r = page - (pre[blockIdx.x] + lo) - (live - moves);
            if (r < done) {
                to = free_page(w, pre, nc, r);
                reinterpret_cast<int2*>(pairs)[r] = make_int2(page, to);
                c.refcounts[to] = ref;
                c.refcounts[page] = 0;
            }
        }
        w.map[page] = to;
    }
}

// One CTA per sequence: its table entries follow the moved pages.
__global__ void __launch_bounds__(kScanThr) pages_rename(const PagesCall c) {
    __shared__ int sums[kWarps];
    pdl_wait_primary();
    const PagesWs w = ws_of(c.workspace, c.num_seqs, c.num_pages);
    const int s = blockIdx.x, tid = threadIdx.x;
    const int L = c.context_lens[s];
    if (L < 0 || L > int64_t(c.max_blocks) * c.page_size) {
        if (tid == 0) flag(c.dev_status, PA_DEV_BAD_LEN);
        return;
    }
    int v = 0;
    for (int i = tid; i < n_chunks(c.num_pages); i += kScanThr) v += w.count[i];
    block_scan(v, sums);
    int live = c.num_pages;
    for (int x = 0; x < kWarps; ++x) live -= sums[x];
    const int used = L / c.page_size + (L % c.page_size != 0);
    int32_t* row = c.block_tables + int64_t(s) * c.max_blocks;
    for (int b = tid; b < used; b += kScanThr) {
        const int pg = row[b];
        if (pg >= live && pg < c.num_pages) row[b] = w.map[pg];
    }
}

// ---- copies ----------------------------------------------------------------------
constexpr int kCopyThr = 256;
constexpr int kCopyPer = 4;  // 16-byte loads of K and of V a thread has in flight

struct CopyArgs {
    const int32_t* pairs;
    uint4* k;
    uint4* v;
    uint32_t* dev_status;
    int64_t page_stride, token_stride, head_stride;  // 16-byte units
    int32_t n, num_pages, parts;                     // parts of a page
    int32_t chunks, row_chunks, head_chunks;         // 16-byte units of a page, a slot, a head
};

// A CTA copies one part of the K and V pages of every step-th pair.
// kFlat: a page is one run of memory.
template <bool kFlat> __global__ void __launch_bounds__(kCopyThr) pages_copy(const CopyArgs a) {
    pdl_wait_primary();
    // The list is read 32 of the CTA's pairs at a time, by every warp: most of
    // one may be empty (a list of 8192 places for 1700 moves took 6 us longer when a
    // CTA read them one by one, a pair ahead).
    const int lane = threadIdx.x & 31;
    const int part = int(blockIdx.x) % a.parts, step = int(gridDim.x) / a.parts;
    const int2* pairs = reinterpret_cast<const int2*>(a.pairs);
    for (int64_t i0 = int(blockIdx.x) / a.parts; i0 < a.n; i0 += int64_t(32) * step) {
        const int64_t mine = i0 + int64_t(lane) * step;
        const int2 read = mine < a.n ? pairs[mine] : make_int2(-1, -1);
        const bool real = read.x >= 0 && read.y >= 0;
        const bool in = real && read.x < a.num_pages && read.y < a.num_pages;
        if (real && !in && threadIdx.x < 32) flag(a.dev_status, PA_DEV_BAD_INDEX);
        for (unsigned m = __ballot_sync(0xffffffffu, in && read.x != read.y); m; m &= m - 1) {
            const int l = __ffs(m) - 1;
            const int2 p = make_int2(__shfl_sync(0xffffffffu, read.x, l), __shfl_sync(0xffffffffu, read.y, l));
            const int c0 = part * (kCopyThr * kCopyPer) + int(threadIdx.x);
            const int64_t from = int64_t(p.x) * a.page_stride, to = int64_t(p.y) * a.page_stride;
            uint4 x[kCopyPer], y[kCopyPer];
            int64_t off[kCopyPer];
#pragma unroll
            for (int i = 0; i < kCopyPer; ++i) {
                const int ch = c0 + i * kCopyThr;
                if (kFlat) {
                    off[i] = ch;
                } else {
                    const int slot = ch / a.row_chunks, in = ch - slot * a.row_chunks;
                    const int head = in / a.head_chunks;
                    off[i] = slot * a.token_stride + head * a.head_stride + (in - head * a.head_chunks);
                }
                if (ch < a.chunks) {
                    x[i] = a.k[from + off[i]];
                    y[i] = a.v[from + off[i]];
                }
            }
#pragma unroll
            for (int i = 0; i < kCopyPer; ++i)
                if (c0 + i * kCopyThr < a.chunks) {
                    a.k[to + off[i]] = x[i];
                    a.v[to + off[i]] = y[i];
                }
        }
    }
}

// ---- store -------------------------------------------------------------------------
constexpr int kStoreThr = 256;

struct StoreArgs {
    const uint4* k;
    const uint4* v;
    const int32_t* row_index;
    uint4* k_cache;
    uint4* v_cache;
    const int32_t* cu_lens;
    const int32_t* block_tables;
    const int32_t* context_lens;
    uint32_t* dev_status;
    int64_t k_stride, v_stride, page_stride, token_stride, head_stride;  // 16-byte units
    int32_t num_seqs, total_rows, max_rows, source_rows, num_pages, max_blocks, page_size;
    int32_t row_chunks, head_chunks;  // 16-byte units of a row, of a head
};

// One warp per destination row.
__global__ void __launch_bounds__(kStoreThr) store_rows(const StoreArgs a) {
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0)  // a sequence without rows of its own is seen by nobody else
        for (int s = threadIdx.x; s < a.num_seqs; s += kStoreThr) {
            const int r0 = a.cu_lens[s], r1 = a.cu_lens[s + 1];
            if (r0 < 0 || r1 < r0 || r1 > a.total_rows || r1 - r0 > a.max_rows) flag(a.dev_status, PA_DEV_BAD_LEN);
        }
    const int row = int(blockIdx.x) * (kStoreThr / 32) + int(threadIdx.x >> 5);
    if (row >= a.total_rows) return;
    // the sequence: the number of ends at or before the row, 32 probes at a time
    int lo = 0, hi = a.num_seqs;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + step * (lane + 1) - 1;  // the last of each of 32 runs
        const int k = __popc(__ballot_sync(0xffffffffu, at < hi && a.cu_lens[at + 1] <= row));
        lo = min(lo + step * k, hi);
        hi = min(hi, lo + step - 1);
    }
    const int s = lo;
    if (s >= a.num_seqs) return;  // behind the last sequence
    const int r0 = a.cu_lens[s], r1 = a.cu_lens[s + 1], L = a.context_lens[s];
    if (row < r0) return;  // before the first sequence (ends out of order are flagged above)
    const int n = r1 - r0;
    if (r0 < 0 || row >= r1 || r1 > a.total_rows || n > a.max_rows || L < n ||
        L > int64_t(a.max_blocks) * a.page_size) {
        if (lane == 0) flag(a.dev_status, PA_DEV_BAD_LEN);
        return;
    }
    const int pos = L - n + (row - r0);
    const int pg = a.block_tables[int64_t(s) * a.max_blocks + pos / a.page_size];
    const int from = a.row_index ? a.row_index[row] : row;
    if (pg < 0 || pg >= a.num_pages || from < 0 || from >= a.source_rows) {
        if (lane == 0) flag(a.dev_status, pg < 0 || pg >= a.num_pages ? PA_DEV_BAD_PAGE : PA_DEV_BAD_INDEX);
        return;
    }
    const uint4* ks = a.k + int64_t(from) * a.k_stride;
    const uint4* vs = a.v + int64_t(from) * a.v_stride;
    const int64_t to = int64_t(pg) * a.page_stride + int64_t(pos % a.page_size) * a.token_stride;
    for (int c0 = lane; c0 < a.row_chunks; c0 += 32 * kCopyPer) {
        uint4 x[kCopyPer], y[kCopyPer];
#pragma unroll
        for (int i = 0; i < kCopyPer; ++i)
            if (c0 + 32 * i < a.row_chunks) {
                x[i] = ks[c0 + 32 * i];
                y[i] = vs[c0 + 32 * i];
            }
#pragma unroll
        for (int i = 0; i < kCopyPer; ++i)
            if (c0 + 32 * i < a.row_chunks) {
                const int head = (c0 + 32 * i) / a.head_chunks;
                const int64_t off = to + head * a.head_stride + (c0 + 32 * i - head * a.head_chunks);
                a.k_cache[off] = x[i];
                a.v_cache[off] = y[i];
            }
    }
}

size_t prefix_bytes(int pages) { return sizeof(int) * size_t(n_chunks(pages)); }

}  // namespace

size_t pages_workspace_bytes(int num_seqs, int num_pages) {
    const size_t wide = size_t(num_seqs) + n_blocks(num_seqs);
    const size_t words = size_t(n_chunks(num_pages)) * (kChunk + 1) + num_pages;
    return (wide * 8 + words * 4 + 255) & ~size_t(255);
}

cudaError_t launch_pages_resize(const PagesCall& c, const int32_t* new_lens, int32_t* pairs, cudaStream_t st) {
    const int scan = n_chunks(c.num_pages) + n_blocks(c.num_seqs);
    cudaError_t e = launch_pdl(pages_scan, dim3(scan), dim3(kScanThr), 0, st, c, new_lens);
    if (e != cudaSuccess) return e;
    return launch_pdl(pages_resize, dim3(c.num_seqs), dim3(kScanThr), prefix_bytes(c.num_pages), st, c, new_lens, pairs);
}

cudaError_t launch_pages_fork(const PagesCall& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t st) {
    return launch_pdl(pages_fork, dim3(n), dim3(kScanThr), 0, st, c, src, dst, n);
}

cudaError_t launch_pages_compact(const PagesCall& c, int32_t* pairs, int max_moves, int32_t* num_moves,
                                 cudaStream_t st) {
    const int nc = n_chunks(c.num_pages);
    cudaError_t e =
        launch_pdl(pages_scan, dim3(nc), dim3(kScanThr), 0, st, c, static_cast<const int32_t*>(nullptr));
    if (e != cudaSuccess) return e;
    e = launch_pdl(pages_compact, dim3(nc), dim3(kScanThr), prefix_bytes(c.num_pages), st, c, pairs, max_moves, num_moves);
    if (e != cudaSuccess) return e;
    return launch_pdl(pages_rename, dim3(c.num_seqs), dim3(kScanThr), 0, st, c);
}

cudaError_t launch_pages_copy(const CacheArgs& c, int Hkv, int D, int elt_bytes, const int32_t* pairs, int n,
                              uint32_t* dev_status, cudaStream_t st) {
    CopyArgs a;
    a.pairs = pairs;
    a.k = static_cast<uint4*>(const_cast<void*>(c.k));
    a.v = static_cast<uint4*>(const_cast<void*>(c.v));
    a.dev_status = dev_status;
    a.page_stride = c.page_stride * elt_bytes / 16;
    a.token_stride = c.token_stride * elt_bytes / 16;
    a.head_stride = c.head_stride * elt_bytes / 16;
    a.n = n;
    a.num_pages = c.num_pages;
    a.head_chunks = D * elt_bytes / 16;
    a.row_chunks = Hkv * a.head_chunks;
    a.chunks = c.page_size * a.row_chunks;
    a.parts = (a.chunks + kCopyThr * kCopyPer - 1) / (kCopyThr * kCopyPer);
    const int ctas = (152 * 8 + a.parts - 1) / a.parts;  // per part: eight CTAs an SM in all
    const int grid = (n < ctas ? n : ctas) * a.parts;
    const bool flat = a.head_stride == a.head_chunks && a.token_stride == a.row_chunks;
    return launch_pdl(flat ? pages_copy<true> : pages_copy<false>, dim3(grid), dim3(kCopyThr), 0, st, a);
}

cudaError_t launch_store(const StoreCall& s, cudaStream_t st) {
    const int eb = s.elt_bytes;
    StoreArgs a;
    a.k = static_cast<const uint4*>(s.k);
    a.v = static_cast<const uint4*>(s.v);
    a.row_index = s.row_index;
    a.k_cache = static_cast<uint4*>(const_cast<void*>(s.c.k));
    a.v_cache = static_cast<uint4*>(const_cast<void*>(s.c.v));
    a.cu_lens = s.r.cu_lens;
    a.block_tables = s.c.block_tables;
    a.context_lens = s.c.context_lens;
    a.dev_status = s.dev_status;
    a.k_stride = s.r.k_stride * eb / 16;
    a.v_stride = s.r.v_stride * eb / 16;
    a.page_stride = s.c.page_stride * eb / 16;
    a.token_stride = s.c.token_stride * eb / 16;
    a.head_stride = s.c.head_stride * eb / 16;
    a.num_seqs = s.r.num_seqs;
    a.total_rows = s.r.total_rows;
    a.max_rows = s.r.max_rows;
    a.source_rows = s.source_rows;
    a.num_pages = s.c.num_pages;
    a.max_blocks = s.c.max_blocks;
    a.page_size = s.c.page_size;
    a.head_chunks = s.D * eb / 16;
    a.row_chunks = s.Hkv * a.head_chunks;
    const int rows = kStoreThr / 32;
    return launch_pdl(store_rows, dim3((s.r.total_rows + rows - 1) / rows), dim3(kStoreThr), 0, st, a);
}

}  // namespace pa
