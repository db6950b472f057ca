// pa_key_weights.cu -- the attention weight that each cached key gathers.
//
//   weights_j <- decay weights_j + sum over (row, head) columns c that see j of
//                2^(s_cj - m_c) / l_c,   s = scale log2(e) q.k
//
// A column's largest score m and sum l are needed before any of its weights,
// so there are two passes over the scores.
//
// Few columns (decoding): K is read once.  The first kernel leaves the scores,
// which are much smaller than K, and each chunk's largest scores and sums in
// the workspace; the second joins the chunks' and turns scores into weights.
// Many columns: the second pass computes the scores again.
#include "pa_device.h"
#include "pa_ptx.cuh"
#include "pa_rows.cuh"
#include "pa_serving.h"

#include <type_traits>

namespace pa {

namespace {

constexpr float kLowest = -3.402823466e38f;  // the running maximum before the first score

struct KwArgs {
    const void* q;
    const void* k;
    const int32_t* cu_lens;
    const int32_t* block_tables;
    const int32_t* context_lens;
    float* weights;
    float2* stats;  // [total_rows][Hq]: a column's largest score and the reciprocal of its sum
    float* scores;  // few columns: [num_seqs][Hkv][max_len][width]
    float2* pieces; // few columns: [num_seqs][Hkv][ceil(max_len / 64)][width], largest score and sum of a chunk
    int32_t width;  // of a key's scores, the columns rounded up to even
    uint32_t* dev_status;
    int64_t q_stride, page_stride, token_stride, head_stride;
    int64_t slots;  // of a block table
    int32_t num_seqs, total_rows, max_rows, num_pages, max_blocks, page_size, page_shift;
    int32_t Hq, Hkv, G, max_len;
    float scale_log2, decay;
};

struct KwSeq {
    int row0, T, L;
    bool bad;
};
__device__ inline KwSeq seq_of(const KwArgs& a, int s) {
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
__device__ inline float reciprocal(float l) { return l == 0.f ? 0.f : 1.f / l; }

__device__ inline void join(float& m, float& l, float m2, float l2) {
    const float top = fmaxf(m, m2);
    l = l * ex2(m - top) + l2 * ex2(m2 - top);
    m = top;
}

// ---- few columns ----------------------------------------------------------------
// Chunks of 64 to 512 keys of a (sequence, kv head), numbered sequence by
// sequence and head by head, are shared out in equal runs of consecutive ones.
// A chunk's keys go in tiles of 16 (a page or half of one) to the CTA's four
// warps.  A lane reads its part of a K row straight into the registers of the
// product's fragments: the dims of a row may come in any order, as long as q's
// come in the same, so that lane c of four takes 16 bytes out of each 64.
constexpr int kFewThr = 128;
constexpr int kFewWarps = kFewThr / 32;
constexpr int kFewCols = 32;   // columns of a (sequence, kv head) at most
constexpr int kFewPerSm = 4;   // CTAs
constexpr int kFoldKeys = kFewThr;

struct Place {
    int s, g, chunk;
    int chunks;  // of each head of the sequence
};

// Chunks of a head of sequence s.
__device__ inline int chunks_of(const KwArgs& a, int s, int keys) {
    if (s >= a.num_seqs) return 0;
    const KwSeq q = seq_of(a, s);
    return q.T > 0 ? (q.L + keys - 1) / keys : 0;
}
// All chunks of the call (whole warp).
__device__ inline int64_t all_chunks(const KwArgs& a, int keys, int lane) {
    int64_t n = 0;
    for (int s = lane; s < a.num_seqs; s += 32) n += int64_t(chunks_of(a, s, keys)) * a.Hkv;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}
// Keys of a chunk: 64, doubled while every CTA keeps two chunks.
__device__ inline int chunk_keys(int64_t chunks64, int ctas) {
    int k = 1;
    while (k < 8 && chunks64 / (2 * k) >= 2 * ctas) k *= 2;
    return 64 * k;
}
// The chunk with a number below all_chunks (whole warp).
__device__ inline Place place_of(const KwArgs& a, int64_t id, int keys, int lane) {
    Place p = {0, 0, 0, 0};
    for (int s0 = 0; s0 < a.num_seqs; s0 += 32) {
        const int n = chunks_of(a, s0 + lane, keys);
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
            p.chunks = __shfl_sync(0xffffffffu, n, l);
            const int64_t in = id - (__shfl_sync(0xffffffffu, v, l) - int64_t(p.chunks) * a.Hkv);
            p.g = int(in / p.chunks);
            p.chunk = int(in - int64_t(p.g) * p.chunks);
            return p;
        }
        id -= __shfl_sync(0xffffffffu, v, 31);
    }
    return p;
}
__device__ inline void next_place(const KwArgs& a, Place& p, int64_t id, int keys, int lane) {
    if (++p.chunk < p.chunks) return;
    p.chunk = 0;
    if (++p.g < a.Hkv) return;
    p = place_of(a, id, keys, lane);
}

// The lane's part of 16 rows: rows r and r + 8 (lane = 4 r + c), of each the
// 16-byte units c, c + 4, c + 8, ...
template <typename T, int D> struct RowPart {
    static constexpr int kUnits = D / (4 * Elt<T>::kVec);
    uint4 lo[kUnits], hi[kUnits];
};
template <typename T, int D>
__device__ inline void load_part(RowPart<T, D>& p, const T* r0, const T* r8, int c) {
#pragma unroll
    for (int i = 0; i < RowPart<T, D>::kUnits; ++i) {
        p.lo[i] = __ldg(reinterpret_cast<const uint4*>(r0) + 4 * i + c);
        p.hi[i] = __ldg(reinterpret_cast<const uint4*>(r8) + 4 * i + c);
    }
}

// Columns as the lane meets them in a product: column 8 n + 2 c and the next.
// 16-bit types: q's fragments in registers; fp32: q in shared memory.
template <typename T, int D, int NT> struct FewQ {
    uint2 b[NT][2 * RowPart<T, D>::kUnits];
    __device__ inline void load(const KwArgs& a, const KwSeq& q, int g, int lane, float*) {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int col = 8 * n + (lane >> 2), t = col / a.G;
            const bool real = t < q.T;
            const uint4* from = reinterpret_cast<const uint4*>(
                static_cast<const T*>(a.q) + (real ? int64_t(q.row0 + t) * a.q_stride + int64_t(g * a.G + col - t * a.G) * D : 0));
#pragma unroll
            for (int i = 0; i < RowPart<T, D>::kUnits; ++i) {
                const uint4 v = real ? __ldg(from + 4 * i + c) : make_uint4(0, 0, 0, 0);
                b[n][2 * i] = make_uint2(v.x, v.y);
                b[n][2 * i + 1] = make_uint2(v.z, v.w);
            }
        }
    }
    // x[n]: rows r and r + 8 of columns 8 n + 2 c, 8 n + 2 c + 1, as the MMA leaves them
    __device__ inline void scores(const RowPart<T, D>& k, const float*, int, float (&x)[NT][4]) const {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
#pragma unroll
        for (int i = 0; i < RowPart<T, D>::kUnits; ++i) {
            const uint32_t a0[4] = {k.lo[i].x, k.hi[i].x, k.lo[i].y, k.hi[i].y};
            const uint32_t a1[4] = {k.lo[i].z, k.hi[i].z, k.lo[i].w, k.hi[i].w};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_16816<std::is_same<T, __nv_bfloat16>::value>(x[n], a0, b[n][2 * i].x, b[n][2 * i].y);
                mma_16816<std::is_same<T, __nv_bfloat16>::value>(x[n], a1, b[n][2 * i + 1].x, b[n][2 * i + 1].y);
            }
        }
    }
};
template <int D, int NT> struct FewQ<float, D, NT> {
    __device__ inline void load(const KwArgs& a, const KwSeq& q, int g, int, float* sq) {
        __syncthreads();
        for (int i = threadIdx.x; i < 8 * NT * (D / 4); i += kFewThr) {
            const int col = i / (D / 4), u = i - col * (D / 4), t = col / a.G;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < q.T)
                v = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + int64_t(q.row0 + t) * a.q_stride +
                                                    int64_t(g * a.G + col - t * a.G) * D)[u];
            reinterpret_cast<float4*>(sq)[i] = v;
        }
        __syncthreads();
    }
    __device__ inline void scores(const RowPart<float, D>& k, const float* sq, int lane, float (&x)[NT][4]) const {
        const int c = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int col = 0; col < 8; ++col) {
                float lo = 0.f, hi = 0.f;
#pragma unroll
                for (int i = 0; i < RowPart<float, D>::kUnits; ++i) {
                    const float4 y = reinterpret_cast<const float4*>(sq)[(8 * n + col) * (D / 4) + 4 * i + c];
                    const float4 u = *reinterpret_cast<const float4*>(&k.lo[i]);
                    const float4 v = *reinterpret_cast<const float4*>(&k.hi[i]);
                    lo = fmaf(u.x, y.x, lo), lo = fmaf(u.y, y.y, lo), lo = fmaf(u.z, y.z, lo), lo = fmaf(u.w, y.w, lo);
                    hi = fmaf(v.x, y.x, hi), hi = fmaf(v.y, y.y, hi), hi = fmaf(v.z, y.z, hi), hi = fmaf(v.w, y.w, hi);
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    lo += __shfl_xor_sync(0xffffffffu, lo, o);
                    hi += __shfl_xor_sync(0xffffffffu, hi, o);
                }
                if (c == col / 2) {  // the lane that holds this column
                    x[n][col % 2] = lo;
                    x[n][2 + col % 2] = hi;
                }
            }
    }
};

template <typename T, int D, int NT> __global__ void __launch_bounds__(kFewThr, kFewPerSm) few_scores(const KwArgs a) {
    extern __shared__ float smem[];  // fp32: the columns' q
    __shared__ float2 joined[kFewWarps][8 * NT];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 3, r = lane >> 2;
    if (blockIdx.x == 0)
        for (int s = tid; s < a.num_seqs; s += kFewThr)
            if (seq_of(a, s).bad) flag(a.dev_status, PA_DEV_BAD_LEN);
    const int64_t n64 = all_chunks(a, 64, lane);
    const int keys = chunk_keys(n64, gridDim.x);
    const int64_t total = keys == 64 ? n64 : all_chunks(a, keys, lane);
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    const int64_t id0 = share * blockIdx.x, id1 = min(total, id0 + share);
    if (id0 >= id1) return;
    Place p = place_of(a, id0, keys, lane);
    FewQ<T, D, NT> qf;
    KwSeq q = {};
    int at_s = -1, at_g = -1;
    for (int64_t id = id0; id < id1; ++id) {
        if (p.s != at_s) q = seq_of(a, p.s);
        if (p.s != at_s || p.g != at_g) qf.load(a, q, p.g, lane, smem);
        at_s = p.s, at_g = p.g;
        const int j0 = p.chunk * keys, n_keys = min(keys, q.L - j0), before = q.L - q.T;
        // the lane-th tile's page
        const int tiles = (n_keys + 15) / 16;
        int my_page = 0;
        if (lane < tiles) {
            my_page = a.block_tables[int64_t(p.s) * a.max_blocks + ((j0 + 16 * lane) >> a.page_shift)];
            if (my_page < 0 || my_page >= a.num_pages) {
                my_page = -1;
                if (warp == 0) flag(a.dev_status, PA_DEV_BAD_PAGE);
            }
        }
        const int64_t unit = int64_t(p.s) * a.Hkv + p.g;
        float* out = a.scores + (unit * a.max_len + j0) * a.width;
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = kLowest, l[n][0] = l[n][1] = 0.f;
        for (int tile = warp; tile < tiles; tile += kFewWarps) {
            const int page = __shfl_sync(0xffffffffu, my_page, tile);
            if (page < 0) continue;  // nothing is read of its scores either
            const T* row = static_cast<const T*>(a.k) + page * a.page_stride +
                           ((j0 + 16 * tile) & (a.page_size - 1)) * a.token_stride + p.g * a.head_stride;
            RowPart<T, D> k;
            load_part<T, D>(k, row + r * a.token_stride, row + (r + 8) * a.token_stride, c);
            float x[NT][4];
            qf.scores(k, smem, lane, x);
            const int j = j0 + 16 * tile + r;
            const bool edge = j0 + 16 * tile + 15 > before;  // some column does not see all of the tile
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (8 * n + 2 * c >= a.width) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float s0 = x[n][i] * a.scale_log2, s1 = x[n][2 + i] * a.scale_log2;
                    if (edge) {
                        const int last = before + (8 * n + 2 * c + i) / a.G;
                        if (j > last) s0 = -INFINITY;
                        if (j + 8 > last) s1 = -INFINITY;
                    }
                    const float top = fmaxf(m[n][i], fmaxf(s0, s1));
                    l[n][i] = l[n][i] * ex2(m[n][i] - top) + ex2(s0 - top) + ex2(s1 - top);
                    m[n][i] = top;
                    x[n][i] = s0, x[n][2 + i] = s1;
                }
                float* to = out + int64_t(16 * tile + r) * a.width + 8 * n + 2 * c;
                if (j < q.L) *reinterpret_cast<float2*>(to) = make_float2(x[n][0], x[n][1]);
                if (j + 8 < q.L) *reinterpret_cast<float2*>(to + 8 * a.width) = make_float2(x[n][2], x[n][3]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    join(m[n][i], l[n][i], __shfl_xor_sync(0xffffffffu, m[n][i], o),
                         __shfl_xor_sync(0xffffffffu, l[n][i], o));
                if (r == 0) joined[warp][8 * n + 2 * c + i] = make_float2(m[n][i], l[n][i]);
            }
        __syncthreads();
        if (tid < a.width) {
            float2 x = joined[0][tid];
            for (int w = 1; w < kFewWarps; ++w) join(x.x, x.y, joined[w][tid].x, joined[w][tid].y);
            a.pieces[(unit * ((a.max_len + 63) / 64) + p.chunk) * a.width + tid] = x;
        }
        __syncthreads();
        if (id + 1 < id1) next_place(a, p, id + 1, keys, lane);
    }
}

// Weights from scores: blocks of 128 keys in equal runs, a key to a thread.
__global__ void __launch_bounds__(kFewThr) few_fold(const KwArgs a, const int ctas) {
    __shared__ float2 joined[kFewWarps][kFewCols];
    __shared__ float2 stats[kFewCols];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int keys = chunk_keys(all_chunks(a, 64, lane), ctas);
    const int64_t total = all_chunks(a, kFoldKeys, lane);
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    const int64_t id0 = share * blockIdx.x, id1 = min(total, id0 + share);
    if (id0 >= id1) return;
    Place p = place_of(a, id0, kFoldKeys, lane);
    KwSeq q = {};
    int at_s = -1, at_g = -1;
    for (int64_t id = id0; id < id1; ++id) {
        if (p.s != at_s) q = seq_of(a, p.s);
        const int64_t unit = int64_t(p.s) * a.Hkv + p.g;
        const int cols = q.T * a.G;
        if (p.s != at_s || p.g != at_g) {
            const int n = (q.L + keys - 1) / keys;
            const float2* from = a.pieces + unit * ((a.max_len + 63) / 64) * a.width;
            float m = kLowest, l = 0.f;
            if (lane < cols)
                for (int i = warp; i < n; i += kFewWarps) {
                    const float2 x = from[int64_t(i) * a.width + lane];
                    join(m, l, x.x, x.y);
                }
            __syncthreads();
            if (lane < cols) joined[warp][lane] = make_float2(m, l);
            __syncthreads();
            if (tid < cols) {
                float2 x = joined[0][tid];
                for (int w = 1; w < kFewWarps; ++w) join(x.x, x.y, joined[w][tid].x, joined[w][tid].y);
                stats[tid] = make_float2(x.x, reciprocal(x.y));
            }
            __syncthreads();
        }
        at_s = p.s, at_g = p.g;
        const int j = p.chunk * kFoldKeys + tid, before = q.L - q.T;
        if (j < q.L) {
            float* to = a.weights + unit * a.slots + j;
            const int pg = a.block_tables[int64_t(p.s) * a.max_blocks + (j >> a.page_shift)];
            float w = 0.f;
            if (pg >= 0 && pg < a.num_pages) {
                const float* x = a.scores + (unit * a.max_len + j) * a.width;
                for (int col = 0; col < cols; col += 2) {
                    const float2 y = *reinterpret_cast<const float2*>(x + col);
                    if (j <= before + col / a.G) w += ex2(y.x - stats[col].x) * stats[col].y;
                    if (col + 1 < cols && j <= before + (col + 1) / a.G)
                        w += ex2(y.y - stats[col + 1].x) * stats[col + 1].y;
                }
            }
            if (a.decay > 0.f && j < before) w += a.decay * *to;
            *to = w;
        }
        if (id + 1 < id1) next_place(a, p, id + 1, kFoldKeys, lane);
    }
}

template <typename T, int D, int NT> cudaError_t launch_few(const KwArgs& a, int ctas, cudaStream_t st) {
    const size_t smem = std::is_same<T, float>::value ? 8 * NT * D * sizeof(float) : 0;  // 16 KB at most
    const cudaError_t e = launch_pdl(few_scores<T, D, NT>, dim3(ctas), dim3(kFewThr), smem, st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(few_fold, dim3(ctas), dim3(kFewThr), 0, st, a, ctas);
}

template <typename T> cudaError_t launch_few_of(const KwArgs& a, int D, int ctas, cudaStream_t st) {
    if (D == 64)
        return a.width <= 8    ? launch_few<T, 64, 1>(a, ctas, st)
               : a.width <= 16 ? launch_few<T, 64, 2>(a, ctas, st)
                               : launch_few<T, 64, 4>(a, ctas, st);
    return a.width <= 8    ? launch_few<T, 128, 1>(a, ctas, st)
           : a.width <= 16 ? launch_few<T, 128, 2>(a, ctas, st)
                           : launch_few<T, 128, 4>(a, ctas, st);
}

// ---- CUDA cores: 64 columns x 64 keys to a tile ---------------------------------
constexpr int kThr = 256;
constexpr int kTile = 64;

template <int D> constexpr size_t tile_smem() { return 2 * kTile * (D + 4) * sizeof(float); }

// Rows of D elements to shared memory as floats; row r from from(r), nullptr: zeros.
template <typename T, int D, typename F> __device__ inline void stage(float* to, F from) {
    constexpr int kVec = Elt<T>::kVec, kUnits = D / kVec;
    for (int i = threadIdx.x; i < kTile * kUnits; i += kThr) {
        const int r = i / kUnits, u = i - r * kUnits;
        const T* p = from(r);
        float x[kVec];
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (p) raw = reinterpret_cast<const uint4*>(p)[u];
        vec_to_f32<T>(raw, x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) to[r * (D + 4) + u * kVec + j] = x[j];
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

template <typename T> __device__ inline const T* key_row(const KwArgs& a, int s, int g, int j, int L) {
    if (j >= L) return nullptr;
    const int pg = a.block_tables[int64_t(s) * a.max_blocks + (j >> a.page_shift)];
    if (pg < 0 || pg >= a.num_pages) return nullptr;
    return static_cast<const T*>(a.k) + pg * a.page_stride + (j & (a.page_size - 1)) * a.token_stride +
           g * a.head_stride;
}
// A column's largest score and sum over the keys that it sees.
template <typename T, int D> __global__ void __launch_bounds__(kThr) kw_stats(const KwArgs a) {
    extern __shared__ float smem[];
    float* sq = smem;
    float* sk = smem + kTile * (D + 4);
    __shared__ int there[kTile];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int s = blockIdx.z, g = blockIdx.y, c0 = int(blockIdx.x) * kTile;
    const KwSeq q = seq_of(a, s);
    if (q.bad && g == 0 && blockIdx.x == 0 && threadIdx.x == 0) flag(a.dev_status, PA_DEV_BAD_LEN);
    const int cols = q.T * a.G;
    if (c0 >= cols) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    stage<T, D>(sq, [&](int r) -> const T* {
        const int c = c0 + r, t = c / a.G;
        if (c >= cols) return nullptr;
        return static_cast<const T*>(a.q) + int64_t(q.row0 + t) * a.q_stride + int64_t(g * a.G + c - t * a.G) * D;
    });
    int last[4];  // the last key that the thread's columns see
    float m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = c0 + ty + 16 * i;
        last[i] = c < cols ? q.L - q.T + c / a.G : -1;
        m[i] = kLowest;
        l[i] = 0.f;
    }
    const int end = q.L - q.T + min(cols - 1, c0 + kTile - 1) / a.G + 1;
    for (int j0 = 0; j0 < end; j0 += kTile) {
        __syncthreads();
        stage<T, D>(sk, [&](int r) { return key_row<T>(a, s, g, j0 + r, q.L); });
        if (tid < kTile) {
            there[tid] = key_row<T>(a, s, g, j0 + tid, q.L) != nullptr;
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
                    const float x = acc[i][j] * a.scale_log2, top = fmaxf(m[i], x);
                    l[i] = l[i] * ex2(m[i] - top) + ex2(x - top);
                    m[i] = top;
                }
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[i], o), l2 = __shfl_xor_sync(0xffffffffu, l[i], o);
            const float top = fmaxf(m[i], m2);
            l[i] = l[i] * ex2(m[i] - top) + l2 * ex2(m2 - top);
            m[i] = top;
        }
        const int c = c0 + ty + 16 * i, t = c / a.G;
        if (tx == 0 && c < cols)
            a.stats[int64_t(q.row0 + t) * a.Hq + g * a.G + c - t * a.G] = make_float2(m[i], reciprocal(l[i]));
    }
}

// What 64 keys gather.
template <typename T, int D> __global__ void __launch_bounds__(kThr) kw_gather(const KwArgs a) {
    extern __shared__ float smem[];
    float* sq = smem;
    float* sk = smem + kTile * (D + 4);
    __shared__ int there[kTile];
    __shared__ float part[16][kTile];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int s = blockIdx.z, g = blockIdx.y, j0 = int(blockIdx.x) * kTile;
    const KwSeq q = seq_of(a, s);
    if (q.T == 0 || j0 >= q.L) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int cols = q.T * a.G, before = q.L - q.T;
    stage<T, D>(sk, [&](int r) { return key_row<T>(a, s, g, j0 + r, q.L); });
    if (tid < kTile) there[tid] = key_row<T>(a, s, g, j0 + tid, q.L) != nullptr;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // the first column that sees key j0
    for (int c0 = max(0, j0 - before) * a.G / kTile * kTile; c0 < cols; c0 += kTile) {
        __syncthreads();
        stage<T, D>(sq, [&](int r) -> const T* {
            const int c = c0 + r, t = c / a.G;
            if (c >= cols) return nullptr;
            return static_cast<const T*>(a.q) + int64_t(q.row0 + t) * a.q_stride + int64_t(g * a.G + c - t * a.G) * D;
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
                if (j0 + key <= before + t && there[key]) sum[j] += ex2(acc[i][j] * a.scale_log2 - st.x) * st.y;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) part[ty][tx + 16 * j] = sum[j];
    __syncthreads();
    if (tid < kTile && j0 + tid < q.L) {
        float w = 0.f;
        for (int i = 0; i < 16; ++i) w += part[i][tid];
        float* to = a.weights + (int64_t(s) * a.Hkv + g) * a.slots + j0 + tid;
        if (a.decay > 0.f && j0 + tid < before) w += a.decay * *to;
        *to = w;
    }
}

template <typename T, int D> cudaError_t launch_tiles(const KwArgs& a, cudaStream_t st) {
    static std::atomic<uint64_t> done_stats{0}, done_gather{0};
    cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kw_stats<T, D>), tile_smem<D>(), done_stats);
    if (e == cudaSuccess)
        e = allow_shared_memory(reinterpret_cast<const void*>(kw_gather<T, D>), tile_smem<D>(), done_gather);
    if (e != cudaSuccess) return e;
    const unsigned ct = unsigned((int64_t(a.max_rows) * a.G + kTile - 1) / kTile);
    e = launch_pdl(kw_stats<T, D>, dim3(ct, a.Hkv, a.num_seqs), dim3(kThr), tile_smem<D>(), st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(kw_gather<T, D>, dim3(unsigned((a.max_len + kTile - 1) / kTile), a.Hkv, a.num_seqs), dim3(kThr),
                      tile_smem<D>(), st, a);
}

}  // namespace

namespace {

size_t rounded(size_t n) { return (n + 255) & ~size_t(255); }
int64_t columns(const KeyWeightsCall& c) { return int64_t(c.r.max_rows) * (c.Hq / c.Hkv); }
int few_width(const KeyWeightsCall& c) { return int(columns(c) + 1) / 2 * 2; }
size_t few_units(const KeyWeightsCall& c) { return size_t(c.r.num_seqs) * c.Hkv; }
size_t few_scores_bytes(const KeyWeightsCall& c) {
    return rounded(few_units(c) * c.max_len * few_width(c) * sizeof(float));
}

}  // namespace

size_t key_weights_workspace_bytes(const KeyWeightsCall& c) {
    if (columns(c) <= kFewCols)
        return few_scores_bytes(c) + rounded(few_units(c) * ((c.max_len + 63) / 64) * few_width(c) * sizeof(float2));
    return rounded(size_t(c.r.total_rows) * c.Hq * sizeof(float2));
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
    if (columns(c) <= kFewCols) {
        const int ctas = c.n_ctas * kFewPerSm;
        if (c.dtype == PA_F32) return launch_few_of<float>(a, c.D, ctas, st);
        return c.dtype == PA_F16 ? launch_few_of<__half>(a, c.D, ctas, st)
                                 : launch_few_of<__nv_bfloat16>(a, c.D, ctas, st);
    }
    if (c.dtype == PA_F32) return c.D == 64 ? launch_tiles<float, 64>(a, st) : launch_tiles<float, 128>(a, st);
    if (c.dtype == PA_F16) return c.D == 64 ? launch_tiles<__half, 64>(a, st) : launch_tiles<__half, 128>(a, st);
    return c.D == 64 ? launch_tiles<__nv_bfloat16, 64>(a, st) : launch_tiles<__nv_bfloat16, 128>(a, st);
}

}  // namespace pa
