// pa_evict.cu -- eviction of the keys that gathered the least attention.
//
// Selection: a CTA for each (sequence, kv head), a cluster of them where a
// block table holds more than a CTA's registers.  A warp holds a run of up to 512
// consecutive weights.  Taken as ordered 32-bit keys, three passes of eleven
// bits find the key of the last one that stays, from histograms in shared memory (the
// cluster's added up), and how many of its equals stay with it.  Then ballots
// number the keys that stay, in order; they leave where they came from and what
// they weigh, which is read again.  The passes themselves read what registers hold,
// and again from memory what is beyond them (tables of more than 131,072 slots); they
// are bound by latency.
//
// Move: key j comes from slot kept[j] >= j, so a cluster of CTAs that has the
// keys of one kv head, of K or of V, can work its way up tile by tile, reading a
// tile before it writes it: what a tile overwrites belongs to keys that it or an
// earlier tile has read.  A tile is 8 CTAs wide, so that a long sequence takes
// few of them (with 4: 87 us instead of 67, eight long prompts, kernels of both
// operations), and a row goes to a cluster for each 128 bytes of it: whole rows of
// 256 took 89 us, columns of 32 or 64 bytes, which need no cluster, 86 and 100, as HBM
// reads scattered short pieces badly.  Two rows a thread instead of four: 72 us
// (one long sequence 31 instead of 26); eight: 67 (23, but four short ones 13.6
// instead of 12.2).
//
// Eight prompts of 10,000 to 16,000 tokens down to 2,048 and more, 8 heads of 128, bf16:
// 67 us for 206 MB, of which 30 at a plain copy's rate.  13 are the selection; the
// move waits for the tiles of the longest sequence, one after another.  The next
// tile's loads before the cluster's wait take 74 registers for 40 and so half the
// CTAs at once: 82 us.  Sequences in the order of their lengths: 59 us, but 1 to 3.5
// more wherever they are alike (sixteen of 300 tokens 29 -> 32).
#include <cooperative_groups.h>

#include "pa_ptx.cuh"
#include "pa_serving.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThr = 1024;
constexpr int kSelWarps = kSelThr / 32;
constexpr int kHeld = 16;                  // weights of a thread
constexpr int kRun = kHeld * kSelThr;      // of a CTA
constexpr int kSelMaxCluster = 8;
constexpr int kDigit = 11;                 // bits of a pass, the last one's fewer
constexpr int kBins = 1 << kDigit;
constexpr int kMoveThr = 256;
constexpr int kMovePer = 4;                // rows of a tile that a thread moves
constexpr int kMoveCluster = 8;
constexpr int kMoveWidth = 8;              // 16-byte units of a row that a cluster moves

// What happens to a sequence.
struct Cut {
    int L, n, first, recent;  // keys before and after; which stay whatever their weight
    bool cut, bad;
};

__device__ inline Cut cut_of(const EvictCall& a, int s) {
    Cut c;
    c.L = a.c.context_lens[s];
    const int keep = a.keep_lens[s];
    c.bad = c.L < 0 || c.L > int64_t(a.c.max_blocks) * a.c.page_size;
    if (c.bad) c.L = 0;
    c.cut = !c.bad && keep >= 0 && keep < c.L;
    c.n = c.cut ? keep : c.L;
    c.recent = min(a.recent, c.n);
    c.first = min(a.first, c.n - c.recent);
    return c;
}

// Order of weights as unsigned numbers; NaN as -infinity, -0 as 0.
__device__ inline uint32_t ordered(float w) {
    if (!(w == w)) w = -INFINITY;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <bool kCluster> __global__ void __launch_bounds__(kSelThr) evict_select(const EvictCall a) {
    __shared__ int hist[kBins];
    __shared__ int sums[2][kSelWarps];
    __shared__ int mine[2];  // keys of the CTA's run that equal the last one; that stay for certain
    __shared__ int found[3]; // a digit, how many keys are still to be chosen among its own, how many it has
    cg::cluster_group cluster = cg::this_cluster();
    const int C = kCluster ? int(cluster.num_blocks()) : 1, rank = kCluster ? int(cluster.block_rank()) : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto sync = [&] {
        if (kCluster)
            cluster.sync();
        else
            __syncthreads();
    };
    pdl_wait_primary();
    pdl_launch_dependents();
    const int unit = int(blockIdx.x) / C;
    const int s = unit / a.Hkv, g = unit - s * a.Hkv;
    Cut c = cut_of(a, s);
    const int64_t slots = int64_t(a.c.max_blocks) * a.c.page_size;
    const float* w = a.weights + unit * slots;
    float* w_out = a.weights_out + unit * slots;
    int32_t* kept = a.kept + unit * slots;
    // the CTA's run, the warp's in it: rows of 32 keys, the first kHeld of them held
    const int run = (c.L + C - 1) / C, lo = min(c.L, rank * run), hi = min(c.L, lo + run);
    const int rows = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32;
    const int j0 = lo + warp * rows * 32 + lane;
    float x[kHeld];
    auto weight_of = [&](int i) { return c.cut && i < rows && j0 + 32 * i < hi ? w[j0 + 32 * i] : 0.f; };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) x[i] = weight_of(i);
    bool held = false;  // a page that would be written has another holder
    if (c.cut && a.refcounts)
        for (int b = c.first / a.c.page_size + tid; b < (c.n + a.c.page_size - 1) / a.c.page_size; b += kSelThr) {
            const int pg = a.c.block_tables[int64_t(s) * a.c.max_blocks + b];
            held |= pg >= 0 && pg < a.c.num_pages && a.refcounts[pg] > 1;
        }
    const bool whole = __syncthreads_or(held) != 0;
    if (whole) c.cut = false, c.n = c.L;
    if (g == 0 && rank == 0 && tid == 0) {
        a.new_lens[s] = c.cut ? c.n : -1;
        if (c.bad) flag(a.dev_status, PA_DEV_BAD_LEN);
        if (whole) flag(a.dev_status, PA_DEV_SHARED_PAGE);
    }
    if (!c.cut) {  // the whole cluster
        for (int j = rank * kSelThr + tid; j < c.L; j += C * kSelThr) {
            kept[j] = j;
            w_out[j] = w[j];
        }
        return;
    }
    // the middle: keys that stay by weight, `want` of them
    const int m0 = c.first, m1 = c.L - c.recent;
    int want = c.n - c.first - c.recent;
    const bool any = want > 0;
    // ordered weights; more than any of them for keys that stay anyway, 0 outside the run
    auto key_of = [&](int i, float v) {
        const int j = j0 + 32 * i;
        return i >= rows || j >= hi ? 0u : j < m0 || j >= m1 ? 0xffffffffu : ordered(v);
    };
    uint32_t keys[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) keys[i] = key_of(i, x[i]);
    // f(row, key) for the warp's rows, whole warp
    auto each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i < rows) f(i, keys[i]);
        for (int i = kHeld; i < rows; ++i) f(i, key_of(i, weight_of(i)));
    };
    uint32_t prefix = 0;  // the leading digits of the last key that stays
    for (int top = 32; top > 0; top -= kDigit) {  // bits top - kDigit .. top - 1
        const int shift = max(0, top - kDigit);
        const uint32_t mask = (1u << (top - shift)) - 1u;
        for (int b = tid; b < kBins; b += kSelThr) hist[b] = 0;
        __syncthreads();
        if (top == 32)
            each([&](int, uint32_t k) {
                if (k + 1u > 1u) atomicAdd(&hist[k >> shift], 1);  // neither 0 nor the largest number
            });
        else
            each([&](int, uint32_t k) {
                if ((k ^ prefix) >> top == 0u) atomicAdd(&hist[(k >> shift) & mask], 1);
            });
        sync();
        // from the largest digit down: where the count reaches `want`; a thread has two digits
        constexpr int kMine = kBins / kSelThr;
        int part[kMine], sum = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int bin = kBins - 1 - (kMine * tid + i);
            part[i] = hist[bin];
            if (kCluster) {
                part[i] = 0;
                for (int r = 0; r < C; ++r) part[i] += cluster.map_shared_rank(hist, r)[bin];
            }
            sum += part[i];
        }
        int v = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        if (lane == 31) sums[0][warp] = v;
        if (tid == 0) found[0] = 0, found[1] = 0;
        __syncthreads();
        int above = v - sum + __reduce_add_sync(0xffffffffu, lane < warp ? sums[0][lane] : 0);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            if (above < want && want <= above + part[i]) {
                found[0] = kBins - 1 - (kMine * tid + i);
                found[1] = want - above;
                found[2] = part[i];
            }
            above += part[i];
        }
        sync();  // the others have read this histogram, the CTA its digit
        prefix |= uint32_t(found[0]) << shift;
        want = found[1];
    }
    // keys above the last one stay, and the first `want` equal to it; none where none is wanted
    const bool all_equal = any && want == found[2];  // all of its equals stay
    if (!any) prefix = 0xfffffffeu;
    int eq = 0, st = 0;  // of the warp
    each([&](int, uint32_t k) {
        eq += k == prefix;
        st += k > prefix;
    });
    eq = __reduce_add_sync(0xffffffffu, eq);
    st = __reduce_add_sync(0xffffffffu, st);
    if (lane == 0) sums[0][warp] = eq, sums[1][warp] = st;
    __syncthreads();
    // before the warp's run, in the CTA: each warp adds up for itself
    int eq_at = lane < warp ? sums[0][lane] : 0, st_at = lane < warp ? sums[1][lane] : 0;
    eq_at = __reduce_add_sync(0xffffffffu, eq_at);
    st_at = __reduce_add_sync(0xffffffffu, st_at);
    if (kCluster) {
        if (tid == kSelThr - 1) mine[0] = eq_at + eq, mine[1] = st_at + st;
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            eq_at += cluster.map_shared_rank(mine, r)[0];
            st_at += cluster.map_shared_rank(mine, r)[1];
        }
    }
    const unsigned below = (1u << lane) - 1u;
    if (all_equal) {
        int at = st_at + eq_at;
        each([&](int i, uint32_t k) {
            const unsigned m = __ballot_sync(0xffffffffu, k >= prefix);
            if (k >= prefix) {
                const int to = at + __popc(m & below);
                kept[to] = j0 + 32 * i;
                w_out[to] = w[j0 + 32 * i];
            }
            at += __popc(m);
        });
    } else {
        each([&](int i, uint32_t k) {
            const unsigned em = __ballot_sync(0xffffffffu, k == prefix), sm = __ballot_sync(0xffffffffu, k > prefix);
            const int eb = eq_at + __popc(em & below), sb = st_at + __popc(sm & below);
            if (k > prefix || (k == prefix && eb < want)) {
                const int to = sb + min(eb, want);
                kept[to] = j0 + 32 * i;
                w_out[to] = w[j0 + 32 * i];
            }
            eq_at += __popc(em);
            st_at += __popc(sm);
        });
    }
    if (kCluster) cluster.sync();  // nobody leaves while another may read its counts
}

struct MoveArgs {
    uint4* k;
    uint4* v;
    int64_t page_stride, token_stride, head_stride;  // 16-byte units
    const int32_t* block_tables;
    const int32_t* kept;
    const int32_t* new_lens;
    uint32_t* dev_status;
    int32_t Hkv, max_blocks, page_size, page_shift, num_pages;
    int32_t parts, width;  // columns of a row, and their 16-byte units
};

__global__ void __cluster_dims__(kMoveCluster, 1, 1) __launch_bounds__(kMoveThr) evict_move(const MoveArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    pdl_wait_primary();
    pdl_launch_dependents();
    const int rank = int(cluster.block_rank());
    int id = int(blockIdx.x) / kMoveCluster;
    const int part = id % a.parts;
    id /= a.parts;
    uint4* pool = id & 1 ? a.v : a.k;
    const int unit = id >> 1, s = unit / a.Hkv, g = unit - s * a.Hkv;
    const int n = a.new_lens[s];
    if (n <= 0) return;  // the whole cluster
    const int32_t* table = a.block_tables + int64_t(s) * a.max_blocks;
    const int32_t* kept = a.kept + unit * (int64_t(a.max_blocks) * a.page_size);
    const int per = kMoveThr / a.width, tile = per * kMovePer * kMoveCluster;
    const int mine = rank * kMovePer * per + int(threadIdx.x) / a.width;  // the thread's first row of a tile
    const int64_t off = g * a.head_stride + part * a.width + int(threadIdx.x) % a.width;
    auto place = [&](int slot) -> int64_t {
        const int pg = table[slot >> a.page_shift];
        if (pg < 0 || pg >= a.num_pages) return -1;
        return pg * a.page_stride + (slot & (a.page_size - 1)) * a.token_stride + off;
    };
    int from[kMovePer];  // where the rows of the next tile come from
    auto look = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kMovePer; ++i) {
            const int j = j0 + mine + i * per;
            from[i] = j < n ? kept[j] : -1;
        }
    };
    look(0);
    for (int j0 = 0; j0 < n; j0 += tile) {
        uint4 x[kMovePer];
        int64_t to[kMovePer];
#pragma unroll
        for (int i = 0; i < kMovePer; ++i) {
            const int j = j0 + mine + i * per;
            to[i] = -1;
            if (from[i] >= 0 && from[i] != j) {
                const int64_t src = place(from[i]);
                to[i] = place(j);
                if (src < 0 || to[i] < 0) {
                    flag(a.dev_status, PA_DEV_BAD_PAGE);
                    to[i] = -1;
                } else {
                    x[i] = pool[src];
                }
            }
        }
        look(j0 + tile);
        cluster.sync();  // the tile is read
#pragma unroll
        for (int i = 0; i < kMovePer; ++i)
            if (to[i] >= 0) pool[to[i]] = x[i];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictCall& c, cudaStream_t st) {
    const int units = c.num_seqs * c.Hkv;
    int size = 1;
    const int64_t slots = int64_t(c.c.max_blocks) * c.c.page_size;
    while (size < kSelMaxCluster && int64_t(size) * kRun < slots) size *= 2;
    cudaError_t e;
    if (size == 1) {
        e = launch_pdl(evict_select<false>, dim3(unsigned(units)), dim3(kSelThr), 0, st, c);
    } else {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(units) * size);
        cfg.blockDim = dim3(kSelThr);
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = size;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, evict_select<true>, c);
    }
    if (e != cudaSuccess) return e;
    MoveArgs a;
    a.k = static_cast<uint4*>(const_cast<void*>(c.c.k));
    a.v = static_cast<uint4*>(const_cast<void*>(c.c.v));
    a.page_stride = c.c.page_stride * c.elt_bytes / 16;
    a.token_stride = c.c.token_stride * c.elt_bytes / 16;
    a.head_stride = c.c.head_stride * c.elt_bytes / 16;
    a.block_tables = c.c.block_tables;
    a.kept = c.kept;
    a.new_lens = c.new_lens;
    a.dev_status = c.dev_status;
    a.Hkv = c.Hkv;
    a.max_blocks = c.c.max_blocks;
    a.page_size = c.c.page_size;
    a.page_shift = c.c.page_size == 16 ? 4 : 5;
    a.num_pages = c.c.num_pages;
    const int row = c.D * c.elt_bytes / 16;  // 16-byte units, a power of two from 8 to 64
    a.width = row < kMoveWidth ? row : kMoveWidth;
    a.parts = row / a.width;
    return launch_pdl(evict_move, dim3(unsigned(units) * 2 * a.parts * kMoveCluster), dim3(kMoveThr), 0, st, a);
}

}  // namespace pa
