// pa_rotate.cu -- norms and rotation of queries and keys, and their store.
//
//   y = x rsqrt(mean(x^2) + eps) w;  (y_a, y_b) -> (c y_a - s y_b, s y_a + c y_b)
//
// One pass over the rows: a warp takes a row, or a part of its heads where
// there are too few rows to fill the GPU, and reads the row's cosines and sines
// once for all of them.  A lane holds 16 dims of a head in two runs of eight,
// chosen so that both dims of a pair are its own (the runs lie rotary_dim / 2
// apart, or beside one another where neighbours turn together): the rotation
// needs no exchange, and a call may write over its input.  Only the norm's sum
// crosses the D / 16 lanes of a head.  Heads go in groups as wide as a warp, q's
// first, then k's and v's; the next groups' loads are in flight while a group is
// turned, in paired fp32 arithmetic (without these two 87 us where it was then 66).
// Each number is rounded once, to the output's type.
//
// Bound by HBM: four documents of 8192 rows, 64/8 heads of 128, bf16, with store,
// move 1418 MB in 239 us (5.9 TB/s, 87% of a plain copy's rate).  Twelve ragged
// chunks, 12,343 rows and 332 MB, take 64 us (5.2 TB/s): the grid's start and end
// weigh more.  Loading before a row's sequence is known was slower (72 and
// 272 us), and so were eight warps a CTA (66 and 240).
#include "pa_pairs.cuh"
#include "pa_ptx.cuh"
#include "pa_rows.cuh"
#include "pa_serving.h"

namespace pa {

namespace {

constexpr int kThr = 128;

struct RotateArgs {
    const uint4* q;
    const uint4* k;
    const uint4* v;
    const uint4* q_weight;
    const uint4* k_weight;
    uint4* q_out;
    uint4* k_out;
    uint4* k_cache;  // nullptr: no store
    uint4* v_cache;
    const float* table;
    const int32_t* positions;
    const int32_t* cu_lens;
    const int32_t* block_tables;
    const int32_t* context_lens;  // nullptr: positions are given and nothing is stored
    uint32_t* dev_status;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // 16-byte units
    int64_t page_stride, token_stride, head_stride;
    int32_t num_seqs, total_rows, max_rows, num_pages, max_blocks, page_size;
    int32_t Hq, Hkv;
    int32_t rot, table_rows, axes, end0, end1;  // pairs below end0 follow axis 0, below end1 axis 1
    int32_t whole;  // both are multiples of eight
    int32_t parts;  // warps of a row
    float eps;
};

template <typename T> __device__ inline void to_f32(const uint4 (&raw)[16 / Elt<T>::kVec], float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 16 / Elt<T>::kVec; ++i) vec_to_f32<T>(raw[i], x + i * Elt<T>::kVec);
}

template <typename T> __device__ inline uint4 pack_vec(const float* x);
template <> __device__ inline uint4 pack_vec<float>(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
template <> __device__ inline uint4 pack_vec<__half>(const float* x) {
    uint4 r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return r;
}
template <> __device__ inline uint4 pack_vec<__nv_bfloat16>(const float* x) {
    uint4 r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return r;
}

template <typename T, int D, bool kMixed> __global__ void __launch_bounds__(kThr) rotate_rows(const RotateArgs a) {
    constexpr int kVec = Elt<T>::kVec;
    constexpr int kRun = 8 / kVec;         // 16-byte units of a run of eight dims
    constexpr int kUnits = 2 * kRun;       // of a lane
    constexpr int kLanes = D / 16;         // lanes of a head
    constexpr int kHeads = 32 / kLanes;    // heads of a warp at a time
    constexpr int kHeadUnits = D / kVec;   // 16-byte units of a head
    constexpr int kAhead = kVec / 4;       // groups whose loads are in flight: 64 bytes a lane
    pdl_wait_primary();
    pdl_launch_dependents();
    if (blockIdx.x == 0) flag_bad_rows(a.cu_lens, a.num_seqs, a.total_rows, a.max_rows, a.dev_status);
    const int lane = threadIdx.x & 31;
    const int64_t unit = int64_t(blockIdx.x) * (kThr / 32) + (threadIdx.x >> 5);
    const int64_t row64 = unit / a.parts;
    if (row64 >= a.total_rows) return;
    const int row = int(row64), part = int(unit - row64 * a.parts);
    const int s = seq_of_row(a.cu_lens, a.num_seqs, row, lane);
    if (s >= a.num_seqs) return;  // behind the last sequence
    const int r0 = a.cu_lens[s], r1 = a.cu_lens[s + 1];
    if (row < r0) return;  // before the first sequence (ends out of order are flagged above)
    const int n = r1 - r0;
    if (bad_rows(r0, r1, a.total_rows, a.max_rows) || row >= r1) return;  // flagged above
    int at = 0;
    if (a.context_lens) {
        const int L = a.context_lens[s];
        if (L < n || (a.k_cache && L > int64_t(a.max_blocks) * a.page_size)) {
            if (lane == 0) flag(a.dev_status, PA_DEV_BAD_LEN);
            return;
        }
        at = L - n + (row - r0);
    }
    // cosines and sines of the lane's eight pairs, the same for every head
    const int sub = lane & (kLanes - 1), half = a.rot / 2;
    const bool turns = sub < a.rot / 16;
    uint64_t cs[4], sn[4];  // of pairs 2 i and 2 i + 1
    int pos[3];
    bool off = false;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        pos[i] = i >= a.axes ? 0 : a.positions ? a.positions[int64_t(i) * a.total_rows + row] : at;
        off |= i < a.axes && a.rot && (pos[i] < 0 || pos[i] >= a.table_rows);
    }
    if (off) {
        if (lane == 0) flag(a.dev_status, PA_DEV_BAD_INDEX);
        return;
    }
    if (turns) {
        if (a.whole) {  // the lane's eight pairs follow one axis
            const int where = 8 * sub < a.end0 ? pos[0] : 8 * sub < a.end1 ? pos[1] : pos[2];
            const float* t = a.table + int64_t(where) * a.rot + 8 * sub;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 c = *reinterpret_cast<const float4*>(t + 4 * i);
                const float4 z = *reinterpret_cast<const float4*>(t + half + 4 * i);
                cs[2 * i] = pairs::pack(c.x, c.y), cs[2 * i + 1] = pairs::pack(c.z, c.w);
                sn[2 * i] = pairs::pack(z.x, z.y), sn[2 * i + 1] = pairs::pack(z.z, z.w);
            }
        } else {
            float c[8], z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int pair = 8 * sub + i;
                const int where = pair < a.end0 ? pos[0] : pair < a.end1 ? pos[1] : pos[2];
                const float* t = a.table + int64_t(where) * a.rot + pair;
                c[i] = t[0];
                z[i] = t[half];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cs[i] = pairs::pack(c[2 * i], c[2 * i + 1]);
                sn[i] = pairs::pack(z[2 * i], z[2 * i + 1]);
            }
        }
    }
    // the lane's two runs of eight dims, in 16-byte units
    const int turning = a.rot / 16;
    const int run0 = kRun * (kMixed ? 2 * sub : turns ? sub : 2 * sub);
    const int run1 = kRun * (kMixed ? 2 * sub + 1 : turns ? sub + turning : 2 * sub + 1);
    // where the row's K and V go
    int64_t slot = -1;
    if (a.k_cache) {
        const int pg = a.block_tables[int64_t(s) * a.max_blocks + at / a.page_size];
        if (pg >= 0 && pg < a.num_pages)
            slot = int64_t(pg) * a.page_stride + int64_t(at % a.page_size) * a.token_stride;
        else if (lane == 0)
            flag(a.dev_status, PA_DEV_BAD_PAGE);
    }
    // groups of heads: q's, k's and, with a store, v's
    const int nq = (a.Hq + kHeads - 1) / kHeads, nk = (a.Hkv + kHeads - 1) / kHeads;
    const int groups = nq + nk + (a.k_cache ? nk : 0), mine = lane / kLanes;
    const int g0 = int(int64_t(groups) * part / a.parts), g1 = int(int64_t(groups) * (part + 1) / a.parts);
    const uint4* qr = a.q + row * a.q_stride;
    const uint4* kr = a.k + row * a.k_stride;
    const uint4* vr = a.v + row * a.v_stride;
    auto fetch = [&](int g, uint4 (&raw)[kUnits]) {
        const int h = (g < nq ? g : g < nq + nk ? g - nq : g - nq - nk) * kHeads + mine;
        if (g < g1 && h < (g < nq ? a.Hq : a.Hkv)) {
            const uint4* from = (g < nq ? qr : g < nq + nk ? kr : vr) + h * kHeadUnits;
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                raw[i] = __ldcs(from + run0 + i);
                raw[kRun + i] = __ldcs(from + run1 + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) raw[i] = make_uint4(0, 0, 0, 0);
        }
    };
    uint4 next[kAhead][kUnits];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(g0 + u, next[u]);
    uint64_t w[8];  // the norm's weights of the kind at hand
    const uint4* held = nullptr;
    for (int base = g0; base < g1; base += kAhead) {
        uint4 now[kAhead][kUnits];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int i = 0; i < kUnits; ++i) now[u][i] = next[u][i];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) fetch(base + kAhead + u, next[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int g = base + u;
            if (g >= g1) break;
            const bool is_q = g < nq, is_k = !is_q && g < nq + nk;
            const int h = (is_q ? g : is_k ? g - nq : g - nq - nk) * kHeads + mine;
            const bool real = h < (is_q ? a.Hq : a.Hkv);
            const uint4* weight = is_q ? a.q_weight : is_k ? a.k_weight : nullptr;
            if (weight != nullptr || (is_q || is_k ? half > 0 : false)) {
                float x[16];
                to_f32<T>(now[u], x);
                uint64_t y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = pairs::pack(x[2 * i], x[2 * i + 1]);
                if (weight) {
                    uint64_t sums = pairs::mul(y[0], y[0]);
#pragma unroll
                    for (int i = 1; i < 8; ++i) sums = pairs::fma(y[i], y[i], sums);
                    const float2 two = pairs::unpack(sums);
                    float sum = two.x + two.y;
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (weight != held) {
                        uint4 wr[kUnits];
                        float wf[16];
#pragma unroll
                        for (int i = 0; i < kRun; ++i) {
                            wr[i] = weight[run0 + i];
                            wr[kRun + i] = weight[run1 + i];
                        }
                        to_f32<T>(wr, wf);
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = pairs::pack(wf[2 * i], wf[2 * i + 1]);
                        held = weight;
                    }
                    const float inv = 1.f / sqrtf(sum * (1.f / D) + a.eps);
                    const uint64_t inv2 = pairs::pack(inv, inv);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = pairs::mul(pairs::mul(y[i], inv2), w[i]);
                }
                if (turns) {
                    if (kMixed) {  // dims 2 i and 2 i + 1 lie in one pair
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 v = pairs::unpack(y[i]);
                            const float2 c = pairs::unpack(cs[i / 2]), z = pairs::unpack(sn[i / 2]);
                            const float cc = i & 1 ? c.y : c.x, ss = i & 1 ? z.y : z.x;
                            y[i] = pairs::pack(v.x * cc - v.y * ss, v.x * ss + v.y * cc);
                        }
                    } else {  // dims 2 i, 2 i + 1 of both runs
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint64_t ya = y[i], yb = y[4 + i];
                            y[i] = pairs::fma(ya, cs[i], pairs::mul(yb, pairs::mul(sn[i], pairs::pack(-1.f, -1.f))));
                            y[4 + i] = pairs::fma(ya, sn[i], pairs::mul(yb, cs[i]));
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 v = pairs::unpack(y[i]);
                    x[2 * i] = v.x, x[2 * i + 1] = v.y;
                }
                if (weight || turns) {  // otherwise the dims are as they were
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) now[u][i] = pack_vec<T>(x + i * kVec);
                }
            }
            if (!real) continue;
            auto put = [&](uint4* to) {
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    to[run0 + i] = now[u][i];
                    to[run1 + i] = now[u][kRun + i];
                }
            };
            if (is_q) put(a.q_out + row * a.q_out_stride + h * kHeadUnits);
            if (is_k && a.k_out) put(a.k_out + row * a.k_out_stride + h * kHeadUnits);
            if (!is_q && slot >= 0) put((is_k ? a.k_cache : a.v_cache) + slot + h * a.head_stride);
        }
    }
}

template <typename T, int D> cudaError_t launch_mixed(const RotateArgs& a, bool mixed, cudaStream_t st) {
    const int64_t warps = int64_t(a.total_rows) * a.parts;
    const dim3 grid(unsigned((warps + kThr / 32 - 1) / (kThr / 32)));
    return launch_pdl(mixed ? rotate_rows<T, D, true> : rotate_rows<T, D, false>, grid, dim3(kThr), 0, st, a);
}
template <typename T> cudaError_t launch_dim(const RotateArgs& a, int D, bool mixed, cudaStream_t st) {
    return D == 64 ? launch_mixed<T, 64>(a, mixed, st) : D == 128 ? launch_mixed<T, 128>(a, mixed, st)
                                                                  : launch_mixed<T, 256>(a, mixed, st);
}

}  // namespace

cudaError_t launch_rotate(const RotateCall& c, cudaStream_t st) {
    const int eb = c.dtype == PA_F32 ? 4 : 2;
    RotateArgs a;
    a.q = static_cast<const uint4*>(c.q);
    a.k = static_cast<const uint4*>(c.k);
    a.v = static_cast<const uint4*>(c.v);
    a.q_weight = static_cast<const uint4*>(c.q_weight);
    a.k_weight = static_cast<const uint4*>(c.k_weight);
    a.q_out = static_cast<uint4*>(c.q_out);
    a.k_out = static_cast<uint4*>(c.k_out);
    a.k_cache = static_cast<uint4*>(const_cast<void*>(c.c.k));
    a.v_cache = static_cast<uint4*>(const_cast<void*>(c.c.v));
    a.table = c.table;
    a.positions = c.positions;
    a.cu_lens = c.r.cu_lens;
    a.block_tables = c.c.block_tables;
    a.context_lens = c.c.context_lens;
    a.dev_status = c.dev_status;
    a.q_stride = c.r.q_stride * eb / 16;
    a.k_stride = c.r.k_stride * eb / 16;
    a.v_stride = c.r.v_stride * eb / 16;
    a.q_out_stride = c.t.q_out_stride * eb / 16;
    a.k_out_stride = c.t.k_out_stride * eb / 16;
    a.page_stride = c.c.page_stride * eb / 16;
    a.token_stride = c.c.token_stride * eb / 16;
    a.head_stride = c.c.head_stride * eb / 16;
    a.num_seqs = c.r.num_seqs;
    a.total_rows = c.r.total_rows;
    a.max_rows = c.r.max_rows;
    a.num_pages = c.c.num_pages;
    a.max_blocks = c.c.max_blocks;
    a.page_size = c.c.page_size;
    a.Hq = c.Hq;
    a.Hkv = c.Hkv;
    a.rot = c.t.rotary_dim;
    a.table_rows = c.t.table_rows;
    a.axes = c.t.axes;
    a.end0 = c.t.axes == 1 ? c.t.rotary_dim / 2 : c.t.sections[0];
    a.end1 = a.end0 + c.t.sections[1];
    a.whole = a.end0 % 8 == 0 && a.end1 % 8 == 0;
    a.eps = c.t.eps;
    // A row to a warp, or to several while the warps are fewer than eight an SM (64
    // rows of 32/8 heads of 128: 4.0 us, one warp a row 5.2; 600 rows 6.8 us, with
    // twice as many warps 9.3, with one a row 9.7).
    const int wide = 512 / c.D;  // heads of a group
    const int groups = (c.Hq + wide - 1) / wide + (c.Hkv + wide - 1) / wide * (a.k_cache ? 2 : 1);
    const int want = (152 * 8 + a.total_rows - 1) / a.total_rows;
    a.parts = want < 1 ? 1 : want > groups ? groups : want;
    return c.dtype == PA_F32   ? launch_dim<float>(a, c.D, c.t.interleaved, st)
           : c.dtype == PA_F16 ? launch_dim<__half>(a, c.D, c.t.interleaved, st)
                               : launch_dim<__nv_bfloat16>(a, c.D, c.t.interleaved, st);
}

}  // namespace pa
