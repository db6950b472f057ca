// pa_packed_f32.cu -- prompt and tree attention with fp32 Q/K/V on the CUDA
// cores, register-tiled.
//
// A tile is 64 distributions (row = token * G + head: 64/G consecutive packed
// rows times the G q heads of one kv head), so every K/V row staged in shared
// memory serves them all.  Keys come in blocks of 64, copied by 16-byte
// cp.async one block ahead: packed rows (prompt; a tree's drafts) or pages
// gathered through the block table (a tree's history).  A thread owns 4 x 4
// scores (4 distributions, 4 keys 16 apart) and the same distributions' rows
// of O (4 or 8 dims); probabilities pass to P.V transposed through shared
// memory.  The softmax is online, in base 2; row maxima and sums go over the
// 16 threads of a row group by shuffles in a fixed order.
//
// What bounds it: the FMA pipes and shared-memory reads (64 FMAs per 8 vector
// loads) on long prompts; the dependent chain of loads on short calls.  fp32
// stays off the tensor cores: one tf32 product keeps 11 bits.
//
// Prompt: one CTA per tile (pa_prompt_plan.cuh), latest rows (most keys) first.  Tree: one CTA per
// share of the keys (pa_tree_plan.cuh).
#include "pa_device.h"
#include "pa_prompt_plan.cuh"
#include "pa_ptx.cuh"
#include "pa_serving.h"
#include "pa_tree_plan.cuh"

#include <type_traits>

namespace pa {

namespace {

constexpr int kM = 64;     // distributions of a tile
constexpr int kKB = 64;    // keys of a block
constexpr int kThr = 256;  // 16 row groups x 16 threads

__device__ inline void cp16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ inline void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ inline void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ inline float group_sum(float v) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ inline float group_max(float v) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <int D> struct Tile {
    static constexpr int kLd = D + 4;    // padded row (floats)
    static constexpr int kQ = kM * kLd;  // Q tile
    static constexpr int kBlk = kKB * kLd;
    static constexpr int kPld = kM + 4;  // row of P transposed: [key][distribution]
    static constexpr size_t kBytes =
        sizeof(float) * (size_t(kQ) + 4 * size_t(kBlk) + size_t(kKB) * kPld) + sizeof(int) * 2 * kKB;
};

template <int D, bool kTree>
__global__ void __launch_bounds__(kThr, 1) packed_f32(const PackedAttn a, const TreeShape shape, const PromptShape prompt, int n_tiles) {
    using S = Tile<D>;
    constexpr int kLd = S::kLd, kPld = S::kPld;
    constexpr int kDv = D / 64;                // float4 columns of O a thread owns
    constexpr int kChunks = D / 4;             // 16-byte chunks of a K/V row
    constexpr int kCp = kKB * kChunks / kThr;  // K (and V) copies a thread issues per block
    extern __shared__ float4 smem4[];
    float* q_s = reinterpret_cast<float*>(smem4);
    float* kv_s = q_s + S::kQ;                             // [2 buffers][K, V][kKB][kLd]
    float* p_t = kv_s + 4 * S::kBlk;                       // [kKB][kPld]
    int* ok_s = reinterpret_cast<int*>(p_t + kKB * kPld);  // [2 buffers][kKB]: key present

    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int G = a.Hq / a.Hkv;
    const int tq = kM / G;  // packed rows of a tile
    pdl_wait_primary();
    pdl_launch_dependents();  // after the wait, so that nothing overtakes what it waited for

    TreeWalk walk;
    TreeItem it;
    // what there is to join here; first that there is nothing
    auto put_join = [&](int4 u) {
        if (tid == 0) tree_joins(a.workspace, kM, D, a.n_ctas)[blockIdx.x] = u;
    };
    if constexpr (kTree) {
        if (blockIdx.x == 0) tree_flag_lengths(shape, a.dev_status);
        walk.start(shape, blockIdx.x);
        const bool any = walk.next(shape, it);
        if (!any || !begins(it)) put_join(make_int4(0, 0, 0, 0));
        if (!any) return;
    } else if (n_tiles == 0) {  // blockIdx.x is the unit's number; every warp finds it
        PromptUnits units;
        units.start(prompt);
        if (blockIdx.x == 0)
            for (int s = tid; s < a.r.num_seqs; s += kThr) {
                const int r0 = a.r.cu_lens[s], r1 = a.r.cu_lens[s + 1];
                if (r0 < 0 || r1 < r0 || r1 > a.r.total_rows || r1 - r0 > a.r.max_rows) flag(a.dev_status, PA_DEV_BAD_LEN);
            }
        if (!units.get(prompt, blockIdx.x, it)) return;
    } else {
        // blockIdx.x = (tile from the last) x (sequence, kv head)
        const int per = a.Hkv * a.r.num_seqs;
        const int u = int(blockIdx.x) % per, tile = n_tiles - 1 - int(blockIdx.x) / per;
        it.g = u % a.Hkv;
        it.seq = u / a.Hkv;
        const int r0 = a.r.cu_lens[it.seq], T = a.r.cu_lens[it.seq + 1] - r0;
        if (r0 < 0 || T < 0 || T > a.r.max_rows || r0 + T > a.r.total_rows) {
            if (tile == 0 && tid == 0) flag(a.dev_status, PA_DEV_BAD_LEN);
            return;
        }
        it.t0 = tile * tq;
        if (it.t0 >= T) return;
        it.n_rows = min(tq, T - it.t0);
        it.row0 = r0 + it.t0;
        it.T = T;
        it.L = it.nh = it.b0 = 0;
        it.b1 = (it.t0 + it.n_rows + kKB - 1) / kKB;
        it.slot = -1;
        it.bad_len = false;
    }

    for (;;) {  // the items of the share (prompt: one)
        if (kTree && begins(it)) put_join(join_of(it));
        const float* kp = static_cast<const float*>(a.k) + int64_t(it.row0 - it.t0) * a.r.k_stride + it.g * D;
        const float* vp = static_cast<const float*>(a.v) + int64_t(it.row0 - it.t0) * a.r.v_stride + it.g * D;
        const float* kc = nullptr;
        const float* vc = nullptr;
        const int32_t* table = nullptr;
        if constexpr (kTree) {
            kc = static_cast<const float*>(a.c.k) + int64_t(it.g) * a.c.head_stride;
            vc = static_cast<const float*>(a.c.v) + int64_t(it.g) * a.c.head_stride;
            table = a.c.block_tables + int64_t(it.seq) * a.c.max_blocks;
        }
        // keys of packed rows that some row of the tile may see
        const int p_end = kTree ? (it.bad_len ? 0 : it.T) : it.t0 + it.n_rows;

        // Block b into buffer u: absent keys become zero rows marked not ok.
        auto load_block = [&](int b, int u) {
            float* ks = kv_s + 2 * u * S::kBlk;
            float* vs = ks + S::kBlk;
            const bool hist = kTree && b < it.nh;
#pragma unroll
            for (int n = 0; n < kCp; ++n) {
                const int i = tid + n * kThr;
                const int j = i / kChunks, c = i % kChunks;
                const float *ksrc = nullptr, *vsrc = nullptr;
                bool ok;
                if (hist) {
                    const int key = b * kKB + j;
                    ok = key < it.L;
                    if (ok) {
                        const int P = a.c.page_size;
                        const int pg = table[key / P];
                        ok = pg >= 0 && pg < a.c.num_pages;
                        if (ok) {
                            const int64_t off =
                                int64_t(pg) * a.c.page_stride + int64_t(key % P) * a.c.token_stride + c * 4;
                            ksrc = kc + off;
                            vsrc = vc + off;
                        } else if (c == 0) {
                            flag(a.dev_status, PA_DEV_BAD_PAGE);
                        }
                    }
                } else {
                    const int key = (b - it.nh) * kKB + j;
                    ok = key < p_end;
                    ksrc = kp + int64_t(key) * a.r.k_stride + c * 4;
                    vsrc = vp + int64_t(key) * a.r.v_stride + c * 4;
                }
                float* kd = ks + j * kLd + c * 4;
                float* vd = vs + j * kLd + c * 4;
                if (ok) {
                    cp16(kd, ksrc);
                    cp16(vd, vsrc);
                } else {
                    *reinterpret_cast<float4*>(kd) = make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4*>(vd) = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (c == 0) ok_s[u * kKB + j] = ok;
            }
            cp_commit();
        };
        load_block(it.b0, 0);  // in flight while q is staged

        for (int i = tid; i < kM * kChunks; i += kThr) {
            const int r = i / kChunks, c = i % kChunks;
            const int t = r / G, h = r - t * G;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < tq * G && t < it.n_rows)
                x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                                     int64_t(it.row0 + t) * a.r.q_stride + (it.g * G + h) * D + c * 4);
            *reinterpret_cast<float4*>(q_s + r * kLd + c * 4) = x;
        }

        // ---- this thread's four distributions --------------------------------------
        bool rok[4];
        int trow[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            trow[i] = r / G;
            rok[i] = r < tq * G && trow[i] < it.n_rows;
        }
        const bool live = (tid >> 5) * 8 < it.n_rows * G;
        float o[4][4 * kDv];
        float m_run[4], l_part[4];  // l_part: this thread's keys only
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m_run[i] = -INFINITY;
            l_part[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 4 * kDv; ++e) o[i][e] = 0.f;
        }

        for (int b = it.b0; b < it.b1; ++b) {
            const int u = (b - it.b0) & 1;
            if (b + 1 < it.b1) {
                load_block(b + 1, u ^ 1);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncthreads();  // block b (and the q tile) in shared memory
            const float* ks = kv_s + 2 * u * S::kBlk;
            const float* vs = ks + S::kBlk;
            const bool hist = kTree && b < it.nh;
            // a packed block that some row of the tile sees only in part
            const bool part = !hist && (kTree || (b + 1) * kKB > it.t0 + 1);

            // ---- scores: s[i][k] = q(ty*4+i) . k(tx+16k), by warps that have a
            // distribution (a small tree fills few of the tile's) ------------------
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
#pragma unroll 4
            for (int d = live ? 0 : D; d < D; d += 4) {
                float4 qv[4], kv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(q_s + (ty * 4 + i) * kLd + d);
#pragma unroll
                for (int k = 0; k < 4; ++k) kv[k] = *reinterpret_cast<const float4*>(ks + (tx + 16 * k) * kLd + d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        s[i][k] = fmaf(qv[i].x, kv[k].x, s[i][k]);
                        s[i][k] = fmaf(qv[i].y, kv[k].y, s[i][k]);
                        s[i][k] = fmaf(qv[i].z, kv[k].z, s[i][k]);
                        s[i][k] = fmaf(qv[i].w, kv[k].w, s[i][k]);
                    }
            }

            // ---- mask, online softmax, P transposed into shared memory -------------
            bool kok[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) kok[k] = ok_s[u * kKB + tx + 16 * k] != 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w0 = 0xffffffffu, w1 = 0xffffffffu;  // the block's 64 keys of this row
                if (part) {
                    if constexpr (kTree) {
                        const int w = (b - it.nh) * 2;
                        const uint32_t* mask = a.tree_mask + int64_t(it.row0 + trow[i]) * a.mask_words;
                        w0 = rok[i] && w < a.mask_words ? mask[w] : 0u;
                        w1 = rok[i] && w + 1 < a.mask_words ? mask[w + 1] : 0u;
                    } else {
                        const int n = rok[i] ? it.t0 + trow[i] + 1 - b * kKB : 0;  // keys seen
                        w0 = n >= 32 ? w0 : n <= 0 ? 0u : (1u << n) - 1u;
                        w1 = n >= 64 ? w1 : n <= 32 ? 0u : (1u << (n - 32)) - 1u;
                    }
                }
                float mb = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // key tx + 16k: words 0, 0, 1, 1
                    const bool see = kok[k] && (((k < 2 ? w0 : w1) >> (tx + 16 * (k & 1))) & 1u);
                    s[i][k] = see ? s[i][k] * a.scale_log2 : -INFINITY;
                    mb = fmaxf(mb, s[i][k]);
                }
                const float m_new = fmaxf(m_run[i], group_max(mb));
                const float base = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: weights 0, not NaN
                const float alpha = ex2(m_run[i] - base);
                float ps = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s[i][k] = ex2(s[i][k] - base);
                    ps += s[i][k];
                }
                l_part[i] = l_part[i] * alpha + ps;
                m_run[i] = m_new;
#pragma unroll
                for (int e = 0; e < 4 * kDv; ++e) o[i][e] *= alpha;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(p_t + (tx + 16 * k) * kPld + ty * 4) =
                    make_float4(s[0][k], s[1][k], s[2][k], s[3][k]);
            __syncthreads();  // P complete

            // ---- O += P V ---------------------------------------------------------
            // In a block seen in part a key of weight 0 is passed over, so that
            // a NaN or infinity in its V stays out of the rows that do not see it.
            auto pv = [&](auto skip_zero) {
#pragma unroll 4
                for (int j = live ? 0 : kKB; j < kKB; ++j) {
                    const float4 p = *reinterpret_cast<const float4*>(p_t + j * kPld + ty * 4);
                    const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                    for (int v = 0; v < kDv; ++v) {
                        const float4 w = *reinterpret_cast<const float4*>(vs + j * kLd + 64 * v + tx * 4);
                        const float wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x = fmaf(pr[i], wd[e], o[i][4 * v + e]);
                                o[i][4 * v + e] = decltype(skip_zero)::value && pr[i] == 0.f ? o[i][4 * v + e] : x;
                            }
                    }
                }
            };
            if (part)
                pv(std::true_type());
            else
                pv(std::false_type());
            __syncthreads();  // buffer u and P are rewritten by the next blocks
        }

        // ---- the whole unit: O / l; a piece: max, sum and O into its slot ------------
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float l = group_sum(l_part[i]);
            if (!rok[i]) continue;
            const int r = ty * 4 + i, h = r - trow[i] * G;
            float* dst = static_cast<float*>(a.out) + (int64_t(it.row0 + trow[i]) * a.Hq + it.g * G + h) * D;
            float inv = l == 0.f ? 0.f : 1.f / l;
            if (kTree && it.slot >= 0) {
                float* slot = static_cast<float*>(a.workspace) + slot_floats(kM, D) * it.slot;
                if (tx == 0) *reinterpret_cast<float2*>(slot + 2 * r) = make_float2(m_run[i], l);
                dst = slot + 2 * kM + r * D;
                inv = 1.f;
            }
#pragma unroll
            for (int v = 0; v < kDv; ++v)
                *reinterpret_cast<float4*>(dst + 64 * v + tx * 4) = make_float4(
                    o[i][4 * v] * inv, o[i][4 * v + 1] * inv, o[i][4 * v + 2] * inv, o[i][4 * v + 3] * inv);
        }
        if constexpr (!kTree) break;
        if (!walk.next(shape, it)) break;
    }
}

template <int D> cudaError_t launch(const PackedAttn& a, cudaStream_t st) {
    const size_t sm = Tile<D>::kBytes;
    const int G = a.Hq / a.Hkv, tq = kM / G;
    static std::atomic<uint64_t> allowed[2] = {};
    cudaError_t e = a.tree_mask ? allow_shared_memory(reinterpret_cast<const void*>(packed_f32<D, true>), sm, allowed[1])
                                : allow_shared_memory(reinterpret_cast<const void*>(packed_f32<D, false>), sm, allowed[0]);
    if (e != cudaSuccess) return e;
    TreeShape s = {};
    if (!a.tree_mask) {
        const int64_t tiles = (int64_t(a.r.max_rows) + tq - 1) / tq, ctas = tiles * a.Hkv * a.r.num_seqs;
        if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
        // A CTA for each tile of each (sequence, kv head), where few of them can be
        // empty; else one for each unit's number, which each CTA takes some time to
        // find, about that of an empty CTA for every 32 sequences (2000 rows and 31
        // prompts of 10, 64/8 heads, 64000 tiles of which 2500 hold rows: 2039 us
        // without numbers, 1864 with).
        const PromptShape numbered = prompt_shape(a, tq, kKB);
        const bool direct = ctas <= prompt_numbers(numbered) * (2 + a.r.num_seqs / 32);
        return launch_pdl(packed_f32<D, false>, dim3(unsigned(direct ? ctas : prompt_numbers(numbered))), dim3(kThr), sm, st,
                          a, s, numbered, direct ? int(tiles) : 0);
    }
    s.cu_lens = a.r.cu_lens;
    s.context_lens = a.c.context_lens;
    s.num_seqs = a.r.num_seqs;
    s.total_rows = a.r.total_rows;
    s.max_rows = a.r.max_rows;
    s.Hkv = a.Hkv;
    s.tu = tq;
    s.tile = 0x7fffffff;  // a unit is one tile: its blocks cost the same
    s.kb = kKB;
    s.start = 1;
    s.min_share = 1;
    s.n_ctas = a.n_ctas;
    s.cap = a.max_history;
    e = launch_pdl(packed_f32<D, true>, dim3(a.n_ctas), dim3(kThr), sm, st, a, s, PromptShape{}, 0);
    if (e != cudaSuccess) return e;
    return launch_join<float, D>(s, a, kM, st);
}

}  // namespace

size_t tree_f32_workspace_bytes(int D, int n_ctas) { return tree_workspace_bytes(kM, D, n_ctas); }

cudaError_t launch_packed_f32(const PackedAttn& a, cudaStream_t st) {
    return a.D == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace pa
