// pa_key_weights.cu -- the attention weight that each cached key gathers.
//
//   weights_j <- decay weights_j + sum over (row, head) columns c that see j of
//                2^(s_cj - m_c) / l_c,   s = scale log2(e) q.k
//
// A column's largest score m and sum l are needed before any of its weights,
// so there are two passes over the scores.
#include "pa_device.h"
#include "pa_ptx.cuh"
#include "pa_rows.cuh"
#include "pa_serving.h"

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
            a.stats[int64_t(q.row0 + t) * a.Hq + g * a.G + c - t * a.G] = make_float2(m[i], 1.f / l[i]);
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

size_t key_weights_workspace_bytes(const KeyWeightsCall& c) {
    return (size_t(c.r.total_rows) * c.Hq * sizeof(float2) + 255) & ~size_t(255);
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
    if (c.dtype == PA_F32) return c.D == 64 ? launch_tiles<float, 64>(a, st) : launch_tiles<float, 128>(a, st);
    if (c.dtype == PA_F16) return c.D == 64 ? launch_tiles<__half, 64>(a, st) : launch_tiles<__half, 128>(a, st);
    return c.D == 64 ? launch_tiles<__nv_bfloat16, 64>(a, st) : launch_tiles<__nv_bfloat16, 128>(a, st);
}

}  // namespace pa
