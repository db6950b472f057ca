// pa_key_weights.cu -- the attention weight that each cached key gathers.
//
//   weights_j <- decay weights_j + sum over (row, head) columns c that see j of
//                2^(s_cj - m_c) / l_c,   s = scale log2(e) q.k
//
// A column's largest score m and sum l are needed before any of its weights,
// so there are two passes over the scores.
//
// Few columns (decoding): K is read once.  The first kernel leaves the scores, and
// each part's largest scores and sums, in the workspace; the second joins the parts'
// and turns scores into weights.  A key's scores are 4 bytes a column out and 4 back:
// with 16-bit types and head_dim 128 a quarter of its K at 8 columns, as much at 32;
// at head_dim 64 twice that share.
// Many columns: the second pass computes the scores again.  The border lies at 32
// columns of a kv head (16 bits, 8 heads of 128; few columns against the tensor cores):
//   8 sequences of 16000: 8 columns 60 against 125 us, 16 78, 32 141
//   one of 3000:          8 columns 8.0 against 19.8 us, 16 10.1, 32 15.9
// In fp32 (4 sequences of 4000, 4 heads) 8 columns take 22 against 119 us, 16 43
// against 121, 32 78 against 128.
#include <cooperative_groups.h>

#include "pa_cp_async.cuh"
#include "pa_device.h"
#include "pa_ptx.cuh"
#include "pa_key_weights.h"

#include <type_traits>

namespace pa {

namespace {

// ---- few columns ----------------------------------------------------------------
// The keys of each (sequence, kv head) in tiles of 16 (a page or half of one),
// numbered sequence by sequence and head by head, are shared out to warps in
// equal runs of consecutive tiles.  A warp leaves its scores, and a piece for
// each head in its run: the columns' largest scores and sums there.  A lane
// takes its part of a K row to the registers of the product's fragments by way
// of slots of shared memory that only it uses, kStages tiles ahead: the dims of
// a row may come in any order, as long as q's come in the same, so that lane c
// of four takes 16 bytes out of each 64.
//
// Eight contexts of 9,999 to 16,384 tokens, 64/8 heads of 128, bf16: 246 MB in 56 us
// (4.4 TB/s, 65% of a plain copy's rate), with scores written and read again; a CTA a
// chunk and K through registers took 101 us.  One token over 3,254: 8.4 us, two
// launches and one round of loads after another (lengths, table, K; pieces, scores).
constexpr int kFewThr = 128;
constexpr int kFewWarps = kFewThr / 32;
constexpr int kFewCols = 32;  // columns of a (sequence, kv head) at most
constexpr int kStages = 3;
constexpr int kMinShare = 4;  // tiles of a warp at least
constexpr int kFoldThr = 128;
constexpr int kFoldPerSm = 8;
constexpr int kFoldKeys = 128;  // the fold's own tile: a key to a thread
constexpr int kFoldAhead = 4;

struct Place {
    int s, g, tile;
    int tiles;  // of each head of the sequence
};

__device__ inline int tiles_of(const KwArgs& a, int s, int keys) {
    if (s >= a.num_seqs) return 0;
    const KwSeq q = kw_seq(a, s);
    return q.T > 0 ? (q.L + keys - 1) / keys : 0;
}
// All tiles of the call (whole warp).
__device__ inline int64_t all_tiles(const KwArgs& a, int keys, int lane) {
    int64_t n = 0;
    for (int s = lane; s < a.num_seqs; s += 32) n += int64_t(tiles_of(a, s, keys)) * a.Hkv;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}
__device__ inline int64_t share_of(int64_t tiles, int workers, int least) {
    const int64_t n = (tiles + workers - 1) / workers;
    return n < least ? least : n;
}
// The tile with a number below all_tiles (whole warp).
__device__ inline Place place_of(const KwArgs& a, int64_t id, int keys, int lane) {
    Place p = {0, 0, 0, 0};
    for (int s0 = 0; s0 < a.num_seqs; s0 += 32) {
        const int n = tiles_of(a, s0 + lane, keys);
        int64_t v = int64_t(n) * a.Hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        const unsigned m = __ballot_sync(0xffffffffu, id < v);
        if (m) {
            const int l = __ffs(m) - 1;
            p.s = s0 + l;
            p.tiles = __shfl_sync(0xffffffffu, n, l);
            const int64_t in = id - (__shfl_sync(0xffffffffu, v, l) - int64_t(p.tiles) * a.Hkv);
            p.g = int(in / p.tiles);
            p.tile = int(in - int64_t(p.g) * p.tiles);
            return p;
        }
        id -= __shfl_sync(0xffffffffu, v, 31);
    }
    return p;
}

template <typename T, int D> struct Few {
    static constexpr int kUnits = D / (4 * Elt<T>::kVec);  // 16-byte units of a lane in a row
    static constexpr int kTileBytes = 16 * D * int(sizeof(T));
    static constexpr size_t kSmem = size_t(kFewWarps) * kStages * kTileBytes;
    static constexpr int kPerSm = kTileBytes <= 4096 ? 4 : 2;  // CTAs: 192 KB of slots an SM at most
};

// q of the columns as the lane meets them in a product, column 8 n + 2 c and
// the next: fragments in registers; fp32 reads q where it lies.
template <typename T, int D, int NT> struct FewQ {
    uint2 b[NT][2 * Few<T, D>::kUnits];
    __device__ inline void load(const KwArgs& a, const KwSeq& q, int g, int lane) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int col = 8 * n + (lane >> 2), t = col / a.G;
            const bool real = t < q.T;
            const uint4* from = reinterpret_cast<const uint4*>(
                static_cast<const T*>(a.q) +
                (real ? int64_t(q.row0 + t) * a.q_stride + int64_t(g * a.G + col - t * a.G) * D : 0));
#pragma unroll
            for (int i = 0; i < Few<T, D>::kUnits; ++i) {
                const uint4 v = real ? __ldg(from + 4 * i + (lane & 3)) : make_uint4(0, 0, 0, 0);
                b[n][2 * i] = make_uint2(v.x, v.y);
                b[n][2 * i + 1] = make_uint2(v.z, v.w);
            }
        }
    }
    // x[n]: rows r and r + 8 of columns 8 n + 2 c, 8 n + 2 c + 1, as the MMA leaves them
    __device__ inline void scores(const uint4* slot, int lane, float (&x)[NT][4]) const {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
#pragma unroll
        for (int i = 0; i < Few<T, D>::kUnits; ++i) {
            const uint4 lo = slot[64 * i + lane], hi = slot[64 * i + 32 + lane];
            const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_16816<std::is_same<T, __nv_bfloat16>::value>(x[n], a0, b[n][2 * i].x, b[n][2 * i].y);
                mma_16816<std::is_same<T, __nv_bfloat16>::value>(x[n], a1, b[n][2 * i + 1].x, b[n][2 * i + 1].y);
            }
        }
    }
};
template <int D, int NT> struct FewQ<float, D, NT> {
    const float* base;
    int64_t stride;
    int G, cols;
    __device__ inline void load(const KwArgs& a, const KwSeq& q, int g, int) {
        base = static_cast<const float*>(a.q) + int64_t(q.row0) * a.q_stride + int64_t(g) * a.G * D;
        stride = a.q_stride;
        G = a.G;
        cols = q.T * a.G;
    }
    __device__ inline void scores(const uint4* slot, int lane, float (&x)[NT][4]) const {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = 8 * n + j;
                float lo = 0.f, hi = 0.f;
                if (col < cols) {
                    const float4* y4 = reinterpret_cast<const float4*>(base + col / G * stride + col % G * D);
#pragma unroll
                    for (int i = 0; i < Few<float, D>::kUnits; ++i) {
                        const float4 y = __ldg(y4 + 4 * i + c);
                        const float4 u = reinterpret_cast<const float4*>(slot)[64 * i + lane];
                        const float4 v = reinterpret_cast<const float4*>(slot)[64 * i + 32 + lane];
                        lo = fmaf(u.x, y.x, lo), lo = fmaf(u.y, y.y, lo), lo = fmaf(u.z, y.z, lo), lo = fmaf(u.w, y.w, lo);
                        hi = fmaf(v.x, y.x, hi), hi = fmaf(v.y, y.y, hi), hi = fmaf(v.z, y.z, hi), hi = fmaf(v.w, y.w, hi);
                    }
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        lo += __shfl_xor_sync(0xffffffffu, lo, o);
                        hi += __shfl_xor_sync(0xffffffffu, hi, o);
                    }
                }
                if (c == j / 2) {  // the lane that holds this column
                    x[n][j % 2] = lo;
                    x[n][2 + j % 2] = hi;
                }
            }
    }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kFewThr, Few<T, D>::kPerSm) few_scores(const KwArgs a) {
    extern __shared__ __align__(16) uint4 slots[];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, r = lane >> 2;
    if (blockIdx.x == 0)
        for (int s = tid; s < a.num_seqs; s += kFewThr)
            if (kw_seq(a, s).bad) flag(a.dev_status, PA_DEV_BAD_LEN);
    const int workers = int(gridDim.x) * kFewWarps;
    // the first CTAs' warps first, so that a small call's warps lie on different SMs
    const int worker = warp * int(gridDim.x) + int(blockIdx.x);
    const int64_t total = all_tiles(a, 16, lane), share = share_of(total, workers, kMinShare);
    const int64_t id1 = min(total, share * (worker + 1));
    int64_t id = share * worker;
    uint4* mine = slots + warp * (kStages * Few<T, D>::kTileBytes / 16);
    const uint32_t mine_u32 = smem_u32(mine);
    const uint64_t policy = l2_policy_evict_first();  // K leaves L2 first: the scores are to be there still
    const bool early = a.max_rows > 1;  // rows that do not see all keys
    while (id < id1) {  // a head's part of the run
        const Place p = place_of(a, id, 16, lane);
        const KwSeq q = kw_seq(a, p.s);
        const int n = int(min(int64_t(p.tiles - p.tile), id1 - id));
        const int64_t unit = int64_t(p.s) * a.Hkv + p.g;
        const int32_t* table = a.block_tables + int64_t(p.s) * a.max_blocks;
        const T* head = static_cast<const T*>(a.k) + p.g * a.head_stride;
        int my_page = 0, page_tile = -32;  // pages of tiles page_tile .. page_tile + 31 of the part, one a lane
        auto page_at = [&](int i) {
            if (i >= page_tile + 32) {
                page_tile = i;
                my_page = -1;
                if (i + lane < n) {
                    my_page = table[(16 * (p.tile + i + lane)) >> a.page_shift];
                    if (my_page < 0 || my_page >= a.num_pages) {
                        my_page = -1;
                        flag(a.dev_status, PA_DEV_BAD_PAGE);
                    }
                }
            }
            return __shfl_sync(0xffffffffu, my_page, i - page_tile);
        };
        uint32_t bad = 0;  // a bit for each tile in flight, the next one lowest: its page is none
        auto fetch = [&](int i) {
            if (i < n) {
                const int page = page_at(i);
                if (page >= 0) {
                    const T* row = head + page * a.page_stride + ((16 * (p.tile + i)) & (a.page_size - 1)) * a.token_stride;
                    const uint4* lo = reinterpret_cast<const uint4*>(row + r * a.token_stride) + c;
                    const uint4* hi = reinterpret_cast<const uint4*>(row + (r + 8) * a.token_stride) + c;
                    const uint32_t to = mine_u32 + (i % kStages) * Few<T, D>::kTileBytes + 16 * lane;
#pragma unroll
                    for (int u = 0; u < Few<T, D>::kUnits; ++u) {
                        cp_async16(to + 1024 * u, lo + 4 * u, policy);
                        cp_async16(to + 1024 * u + 512, hi + 4 * u, policy);
                    }
                } else {
                    bad |= 1u << (i % kStages);
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i);
        FewQ<T, D, NT> qf;
        qf.load(a, q, p.g, lane);
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) m[x][0] = m[x][1] = kLowestScore, l[x][0] = l[x][1] = 0.f;
        const int before = q.L - q.T;
        for (int i = 0; i < n; ++i) {
            fetch(i + kStages - 1);
            cp_wait<kStages - 1>();
            const uint32_t bit = 1u << (i % kStages);
            if (bad & bit) {  // nothing is read of its scores either
                bad &= ~bit;
                continue;
            }
            float x[NT][4];
            qf.scores(mine + (i % kStages) * (Few<T, D>::kTileBytes / 16), lane, x);
            const int j = 16 * (p.tile + i) + r;
            const bool edge = 16 * (p.tile + i) + 15 > before;  // some column does not see all of the tile
            float* to = a.scores + (unit * a.max_len + j) * a.width + 2 * c;
#pragma unroll
            for (int y = 0; y < NT; ++y) {
                if (8 * y + 2 * c >= a.width) continue;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // rounded here, as the fold reads them: not to be contracted with a difference
                    float s0 = __fmul_rn(x[y][k], a.scale_log2), s1 = __fmul_rn(x[y][2 + k], a.scale_log2);
                    if (edge) {
                        const int last = before + (early ? (8 * y + 2 * c + k) / a.G : 0);
                        if (j > last) s0 = -INFINITY;
                        if (j + 8 > last) s1 = -INFINITY;
                    }
                    const float top = fmaxf(m[y][k], fmaxf(s0, s1));
                    l[y][k] = l[y][k] * ex2(m[y][k] - top) + ex2(s0 - top) + ex2(s1 - top);
                    m[y][k] = top;
                    x[y][k] = s0, x[y][2 + k] = s1;
                }
                if (j < q.L) *reinterpret_cast<float2*>(to + 8 * y) = make_float2(x[y][0], x[y][1]);
                if (j + 8 < q.L) *reinterpret_cast<float2*>(to + 8 * (a.width + y)) = make_float2(x[y][2], x[y][3]);
            }
        }
        cp_wait<0>();
        // the piece's number in its head: the workers' that begin before it there
        const int64_t first = id - p.tile;
        const int64_t piece = worker - first / share;
        float2* out = a.pieces + (unit * a.max_pieces + piece) * a.width + 2 * c;
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    kw_join(m[y][k], l[y][k], __shfl_xor_sync(0xffffffffu, m[y][k], o),
                         __shfl_xor_sync(0xffffffffu, l[y][k], o));
                if (r == 0 && 8 * y + 2 * c < a.width) out[8 * y + k] = make_float2(m[y][k], l[y][k]);
            }
        id += n;
    }
}

// Weights from scores: tiles of 128 keys in equal runs, a key to a thread and
// kFoldAhead tiles at a time.  NP pairs of columns.
template <int NP> __global__ void __launch_bounds__(kFoldThr) few_fold(const KwArgs a, const int workers) {
    __shared__ float2 joined[kFoldThr / 32][kFewCols];
    __shared__ float2 stats[2 * NP];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the lengths were there before the scores' kernel let this one start
    const int64_t fine = all_tiles(a, 16, lane), fine_share = share_of(fine, workers, kMinShare);
    const int64_t total = all_tiles(a, kFoldKeys, lane), share = share_of(total, gridDim.x, 1);
    const int64_t id1 = min(total, share * (blockIdx.x + 1));
    bool waited = false;
    for (int64_t id = share * blockIdx.x; id < id1;) {
        const Place p = place_of(a, id, kFoldKeys, lane);
        const KwSeq q = kw_seq(a, p.s);
        const int n = int(min(int64_t(p.tiles - p.tile), id1 - id));
        const int64_t unit = int64_t(p.s) * a.Hkv + p.g;
        const int cols = q.T * a.G, before = q.L - q.T;
        // the head's pieces: of the workers that its first and its last tile belong to, and those between
        int64_t first = 0;
        {
            int64_t sum = 0;
            for (int s = lane; s < p.s; s += 32) sum += int64_t(tiles_of(a, s, 16)) * a.Hkv;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            first = sum + int64_t(p.g) * ((q.L + 15) / 16);
        }
        const int pieces = int((first + (q.L + 15) / 16 - 1) / fine_share - first / fine_share) + 1;
        if (!waited) {
            pdl_wait_primary();
            pdl_launch_dependents();
            waited = true;
        }
        const float2* from = a.pieces + unit * a.max_pieces * a.width;
        float m = kLowestScore, l = 0.f;
        if (lane < cols)
            for (int i = warp; i < pieces; i += kFoldThr / 32) {
                const float2 x = from[int64_t(i) * a.width + lane];
                kw_join(m, l, x.x, x.y);
            }
        __syncthreads();
        if (lane < cols) joined[warp][lane] = make_float2(m, l);
        __syncthreads();
        if (tid < 2 * NP) {
            float2 x = tid < cols ? joined[0][tid] : make_float2(0.f, 0.f);
            if (tid < cols)
                for (int w = 1; w < kFoldThr / 32; ++w) kw_join(x.x, x.y, joined[w][tid].x, joined[w][tid].y);
            stats[tid] = make_float2(x.x, kw_reciprocal(x.y));
        }
        __syncthreads();
        float2 st[2 * NP];
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) st[i] = stats[i];
        const float* x0 = a.scores + unit * a.max_len * a.width;
        float* w0 = a.weights + unit * a.slots;
        const int32_t* table = a.block_tables + int64_t(p.s) * a.max_blocks;
        for (int i = 0; i < n; i += kFoldAhead) {
            float2 x[kFoldAhead][NP];
            float old[kFoldAhead];
            int page[kFoldAhead];
#pragma unroll
            for (int u = 0; u < kFoldAhead; ++u) {
                const int j = (p.tile + i + u) * kFoldKeys + tid;
                const bool in = i + u < n && j < q.L;
                page[u] = in ? table[j >> a.page_shift] : -1;
                old[u] = in && a.decay > 0.f && j < before ? w0[j] : 0.f;
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    x[u][k] = in && 2 * k < a.width
                                  ? *reinterpret_cast<const float2*>(x0 + int64_t(j) * a.width + 2 * k)
                                  : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < kFoldAhead; ++u) {
                const int j = (p.tile + i + u) * kFoldKeys + tid;
                if (i + u >= n || j >= q.L) continue;
                float w = 0.f;
                if (page[u] >= 0 && page[u] < a.num_pages) {
                    const int sees = (j - before) * a.G;  // the columns from this one on see the key
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        if (2 * k < cols && 2 * k >= sees) w += ex2(x[u][k].x - st[2 * k].x) * st[2 * k].y;
                        if (2 * k + 1 < cols && 2 * k + 1 >= sees) w += ex2(x[u][k].y - st[2 * k + 1].x) * st[2 * k + 1].y;
                    }
                }
                w0[j] = w + a.decay * old[u];
            }
        }
        id += n;
    }
    if (!waited) pdl_wait_primary();  // nor may the kernel behind this one start early
}

template <typename T, int D, int NT> cudaError_t launch_few(const KwArgs& a, int sms, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e =
        allow_shared_memory(reinterpret_cast<const void*>(few_scores<T, D, NT>), Few<T, D>::kSmem, done);
    if (e != cudaSuccess) return e;
    const int ctas = sms * Few<T, D>::kPerSm, workers = ctas * kFewWarps;
    e = launch_pdl(few_scores<T, D, NT>, dim3(ctas), dim3(kFewThr), Few<T, D>::kSmem, st, a);
    if (e != cudaSuccess) return e;
    const dim3 grid(sms * kFoldPerSm), block(kFoldThr);
    switch (a.width / 2) {
        case 1: return launch_pdl(few_fold<1>, grid, block, 0, st, a, workers);
        case 2: return launch_pdl(few_fold<2>, grid, block, 0, st, a, workers);
        case 3: return launch_pdl(few_fold<3>, grid, block, 0, st, a, workers);
        case 4: return launch_pdl(few_fold<4>, grid, block, 0, st, a, workers);
        default: return a.width <= 16 ? launch_pdl(few_fold<8>, grid, block, 0, st, a, workers)
                                      : launch_pdl(few_fold<16>, grid, block, 0, st, a, workers);
    }
}

template <typename T> cudaError_t launch_few_of(const KwArgs& a, int D, int sms, cudaStream_t st) {
    if (D == 64)
        return a.width <= 8    ? launch_few<T, 64, 1>(a, sms, st)
               : a.width <= 16 ? launch_few<T, 64, 2>(a, sms, st)
                               : launch_few<T, 64, 4>(a, sms, st);
    return a.width <= 8    ? launch_few<T, 128, 1>(a, sms, st)
           : a.width <= 16 ? launch_few<T, 128, 2>(a, sms, st)
                           : launch_few<T, 128, 4>(a, sms, st);
}

// ---- many columns, fp32: CUDA cores, 64 columns x 64 keys to a tile ---------------------------------
// A cluster of CTAs to 64 columns, or to 64 keys, where there are fewer than two CTAs an
// SM without it: they take the tiles in turn, and the first one joins what they
// found, in order (four sequences of 4000 keys, 40 columns on 4 kv heads: 132 us, one CTA
// each 493; a prompt of 500 rows, 32/4 heads, 170 and 546).  Bound by shared memory's
// reads: eight of 16 bytes for 64 multiply-adds of a thread.
namespace cg = cooperative_groups;

constexpr int kThr = 256;
constexpr int kTile = 64;
constexpr int kTileCluster = 8;

template <int D> constexpr size_t tile_smem() { return 2 * kTile * (D + 4) * sizeof(float); }

// Rows of D elements to shared memory; row r from from(r), nullptr: zeros.
template <int D, typename F> __device__ inline void stage(float* to, F from) {
    constexpr int kUnits = D / 4;
    for (int i = threadIdx.x; i < kTile * kUnits; i += kThr) {
        const int r = i / kUnits, u = i - r * kUnits;
        const float* p = from(r);
        *reinterpret_cast<float4*>(to + r * (D + 4) + u * 4) =
            p ? reinterpret_cast<const float4*>(p)[u] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// acc[i][j] = column (ty + 16 i) . key (tx + 16 j)
template <int D> __device__ inline void products(const float* sq, const float* sk, int tx, int ty, float (&acc)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = *reinterpret_cast<const float4*>(sq + (ty + 16 * i) * (D + 4) + d);
            y[i] = *reinterpret_cast<const float4*>(sk + (tx + 16 * i) * (D + 4) + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
    }
}

__device__ inline const float* key_row(const KwArgs& a, int s, int g, int j, int L) {
    if (j >= L) return nullptr;
    const int pg = a.block_tables[int64_t(s) * a.max_blocks + (j >> a.page_shift)];
    if (pg < 0 || pg >= a.num_pages) return nullptr;
    return static_cast<const float*>(a.k) + pg * a.page_stride + (j & (a.page_size - 1)) * a.token_stride +
           g * a.head_stride;
}
// A column's largest score and sum over the keys that it sees.
template <int D> __global__ void __launch_bounds__(kThr) kw_stats(const KwArgs a) {
    extern __shared__ float smem[];
    float* sq = smem;
    float* sk = smem + kTile * (D + 4);
    __shared__ int there[kTile];
    __shared__ float2 found[kTile];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    pdl_wait_primary();
    pdl_launch_dependents();
    const int s = blockIdx.z, g = blockIdx.y, c0 = int(blockIdx.x) / C * kTile;
    const KwSeq q = kw_seq(a, s);
    if (q.bad && g == 0 && blockIdx.x == 0 && threadIdx.x == 0) flag(a.dev_status, PA_DEV_BAD_LEN);
    const int cols = q.T * a.G;
    if (c0 >= cols) return;  // the whole cluster
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    stage<D>(sq, [&](int r) -> const float* {
        const int c = c0 + r, t = c / a.G;
        if (c >= cols) return nullptr;
        return static_cast<const float*>(a.q) + int64_t(q.row0 + t) * a.q_stride + int64_t(g * a.G + c - t * a.G) * D;
    });
    int last[4];  // the last key that the thread's columns see
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = c0 + ty + 16 * i;
        last[i] = c < cols ? q.L - q.T + c / a.G : -1;
        m[i] = kLowestScore;
        l[i] = 0.f;
    }
    const int end = q.L - q.T + min(cols - 1, c0 + kTile - 1) / a.G + 1;
    for (int j0 = rank * kTile; j0 < end; j0 += C * kTile) {
        __syncthreads();
        stage<D>(sk, [&](int r) { return key_row(a, s, g, j0 + r, q.L); });
        if (tid < kTile) {
            there[tid] = key_row(a, s, g, j0 + tid, q.L) != nullptr;
            if (!there[tid] && j0 + tid < q.L) flag(a.dev_status, PA_DEV_BAD_PAGE);
        }
        __syncthreads();
        float acc[4][4];
        products<D>(sq, sk, tx, ty, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = tx + 16 * j;
                if (j0 + key <= last[i] && there[key]) {
                    const float x = __fmul_rn(acc[i][j], a.scale_log2), top = fmaxf(m[i], x);  // rounded, in both kernels
                    l[i] = l[i] * ex2(m[i] - top) + ex2(x - top);
                    m[i] = top;
                }
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            kw_join(m[i], l[i], __shfl_xor_sync(0xffffffffu, m[i], o), __shfl_xor_sync(0xffffffffu, l[i], o));
        if (tx == 0) found[ty + 16 * i] = make_float2(m[i], l[i]);
    }
    cluster.sync();
    const int c = c0 + tid, t = c / a.G;
    if (rank == 0 && tid < kTile && c < cols) {
        float2 x = found[tid];
        for (int i = 1; i < C; ++i) {
            const float2 y = cluster.map_shared_rank(found, i)[tid];
            kw_join(x.x, x.y, y.x, y.y);
        }
        a.stats[int64_t(q.row0 + t) * a.Hq + g * a.G + c - t * a.G] = make_float2(x.x, kw_reciprocal(x.y));
    }
    cluster.sync();  // nobody leaves while another may read what it found
}

// What 64 keys gather.
template <int D> __global__ void __launch_bounds__(kThr) kw_gather(const KwArgs a) {
    extern __shared__ float smem[];
    float* sq = smem;
    float* sk = smem + kTile * (D + 4);
    __shared__ int there[kTile];
    __shared__ float part[16][kTile];
    __shared__ float found[kTile];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    pdl_wait_primary();
    pdl_launch_dependents();
    const int s = blockIdx.z, g = blockIdx.y, j0 = int(blockIdx.x) / C * kTile;
    const KwSeq q = kw_seq(a, s);
    if (q.T == 0 || j0 >= q.L) return;  // the whole cluster
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int cols = q.T * a.G, before = q.L - q.T;
    stage<D>(sk, [&](int r) { return key_row(a, s, g, j0 + r, q.L); });
    if (tid < kTile) there[tid] = key_row(a, s, g, j0 + tid, q.L) != nullptr;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // the first column that sees key j0
    const int first = max(0, j0 - before) * a.G / kTile * kTile;
    for (int c0 = first + rank * kTile; c0 < cols; c0 += C * kTile) {
        __syncthreads();
        stage<D>(sq, [&](int r) -> const float* {
            const int c = c0 + r, t = c / a.G;
            if (c >= cols) return nullptr;
            return static_cast<const float*>(a.q) + int64_t(q.row0 + t) * a.q_stride + int64_t(g * a.G + c - t * a.G) * D;
        });
        __syncthreads();
        float acc[4][4];
        products<D>(sq, sk, tx, ty, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + ty + 16 * i, t = c / a.G;
            if (c >= cols) continue;
            const float2 st = a.stats[int64_t(q.row0 + t) * a.Hq + g * a.G + c - t * a.G];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = tx + 16 * j;
                if (j0 + key <= before + t && there[key]) sum[j] += ex2(__fmul_rn(acc[i][j], a.scale_log2) - st.x) * st.y;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) part[ty][tx + 16 * j] = sum[j];
    __syncthreads();
    if (tid < kTile) {
        float w = 0.f;
        for (int i = 0; i < 16; ++i) w += part[i][tid];
        found[tid] = w;
    }
    cluster.sync();
    if (rank == 0 && tid < kTile && j0 + tid < q.L) {
        float w = found[tid];
        for (int i = 1; i < C; ++i) w += cluster.map_shared_rank(found, i)[tid];
        float* to = a.weights + (int64_t(s) * a.Hkv + g) * a.slots + j0 + tid;
        if (a.decay > 0.f && j0 + tid < before) w += a.decay * *to;
        *to = w;
    }
    cluster.sync();  // nobody leaves while another may read what it found
}

// A cluster to each of `tiles` tiles of every head.
cudaError_t launch_clusters(void (*kern)(KwArgs), const KwArgs& a, int64_t tiles, int64_t others, int sms, size_t smem,
                            cudaStream_t st) {
    const int64_t heads = int64_t(a.Hkv) * a.num_seqs;
    int size = 1;
    while (size < kTileCluster && size < others && tiles * heads * size < 2 * sms) size *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(tiles * size), a.Hkv, a.num_seqs);
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D> cudaError_t launch_tiles(const KwArgs& a, int sms, cudaStream_t st) {
    static std::atomic<uint64_t> done_stats{0}, done_gather{0};
    cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kw_stats<D>), tile_smem<D>(), done_stats);
    if (e == cudaSuccess)
        e = allow_shared_memory(reinterpret_cast<const void*>(kw_gather<D>), tile_smem<D>(), done_gather);
    if (e != cudaSuccess) return e;
    const int64_t columns = (int64_t(a.max_rows) * a.G + kTile - 1) / kTile, keys = (a.max_len + kTile - 1) / kTile;
    e = launch_clusters(kw_stats<D>, a, columns, keys, sms, tile_smem<D>(), st);
    return e == cudaSuccess ? launch_clusters(kw_gather<D>, a, keys, columns, sms, tile_smem<D>(), st) : e;
}

}  // namespace

namespace {

size_t rounded(size_t n) { return (n + 255) & ~size_t(255); }
int64_t columns(const KeyWeightsCall& c) { return int64_t(c.r.max_rows) * (c.Hq / c.Hkv); }
int few_width(const KeyWeightsCall& c) { return int(columns(c) + 1) / 2 * 2; }
size_t few_units(const KeyWeightsCall& c) { return size_t(c.r.num_seqs) * c.Hkv; }
// Parts of a head: of kMinShare tiles at least, but for the first and the last.
size_t few_pieces(const KeyWeightsCall& c) { return size_t((c.max_len + 15) / 16) / kMinShare + 2; }
size_t stats_bytes(const KeyWeightsCall& c) { return rounded(size_t(c.r.total_rows) * c.Hq * sizeof(float2)); }
size_t few_scores_bytes(const KeyWeightsCall& c) {
    return rounded(few_units(c) * c.max_len * few_width(c) * sizeof(float));
}

}  // namespace

size_t key_weights_workspace_bytes(const KeyWeightsCall& c) {
    if (columns(c) <= kFewCols)
        return few_scores_bytes(c) + rounded(few_units(c) * few_pieces(c) * few_width(c) * sizeof(float2));
    return stats_bytes(c) + (c.dtype == PA_F32 ? 0 : rounded(key_weights_tc_parts(c.n_ctas)));
}

cudaError_t launch_key_weights(const KeyWeightsCall& c, cudaStream_t st) {
    KwArgs a;
    a.q = c.q;
    a.k = c.c.k;
    a.cu_lens = c.r.cu_lens;
    a.block_tables = c.c.block_tables;
    a.context_lens = c.c.context_lens;
    a.weights = c.weights;
    a.stats = static_cast<float2*>(c.workspace);
    a.scores = static_cast<float*>(c.workspace);
    a.pieces = reinterpret_cast<float2*>(static_cast<char*>(c.workspace) + (columns(c) <= kFewCols ? few_scores_bytes(c) : 0));
    a.width = columns(c) <= kFewCols ? few_width(c) : 0;
    a.max_pieces = int64_t(few_pieces(c));
    a.dev_status = c.dev_status;
    a.q_stride = c.r.q_stride;
    a.page_stride = c.c.page_stride;
    a.token_stride = c.c.token_stride;
    a.head_stride = c.c.head_stride;
    a.slots = int64_t(c.c.max_blocks) * c.c.page_size;
    a.num_seqs = c.r.num_seqs;
    a.total_rows = c.r.total_rows;
    a.max_rows = c.r.max_rows;
    a.num_pages = c.c.num_pages;
    a.max_blocks = c.c.max_blocks;
    a.page_size = c.c.page_size;
    a.page_shift = c.c.page_size == 16 ? 4 : 5;
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.G = c.Hq / c.Hkv;
    a.max_len = c.max_len;
    a.scale_log2 = c.scale_log2;
    a.decay = c.decay;
    a.debug_timeout = c.debug_timeout;
    if (columns(c) <= kFewCols) {
        if (c.dtype == PA_F32) return launch_few_of<float>(a, c.D, c.n_ctas, st);
        return c.dtype == PA_F16 ? launch_few_of<__half>(a, c.D, c.n_ctas, st)
                                 : launch_few_of<__nv_bfloat16>(a, c.D, c.n_ctas, st);
    }
    if (c.dtype == PA_F32) return c.D == 64 ? launch_tiles<64>(a, c.n_ctas, st) : launch_tiles<128>(a, c.n_ctas, st);
    return launch_key_weights_tc(a, c.dtype, c.D, c.n_ctas, static_cast<char*>(c.workspace) + stats_bytes(c), st);
}

}  // namespace pa
