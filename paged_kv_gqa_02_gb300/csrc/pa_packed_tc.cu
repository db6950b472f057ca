// pa_packed_tc.cu -- prompt and tree attention for 16-bit Q/K/V on the
// 5th-generation tensor cores (tcgen05 MMA, accumulators in tensor memory,
// operands staged by TMA).  head_dim 64 or 128.
//
// A unit of work is up to 2 x 128 MMA rows of one (sequence, kv head): row tiles
// A and B, each 128/G consecutive packed rows times the G q heads (MMA row =
// token * G + head), against key tiles of 128.  Every K/V tile in shared
// memory serves both row tiles and all G heads.  A unit that fills one row
// tile only is worked on by both sides all the same: side A takes the even key
// tiles and side B the odd ones, each with its own O, max and sum, and the
// epilogue joins them ("twin").  CTAs are persistent, one per SM, and work
// through units or, for a tree, pieces of units:
//   prompt: units in descending order of their key tiles (pa_prompt_plan.cuh
//           beyond 32 sequences), taken one by one;
//           keys are the packed rows 0..t of the unit's own sequence;
//   tree:   the CTA's share of the keys (pa_tree_plan.cuh); key tiles are the
//           history's pages first, then the packed drafts under their mask.
//
// Warp roles, joined by mbarriers; each role walks the items on its own clock,
// so one item's loads and first products run under the last one's softmax and
// epilogue:
//   warps 0-3, 4-7  softmax of side A and of side B: a thread per MMA row
//                   (tensor-memory lane), probabilities written over their
//                   scores, epilogue
//   warp 8          finds the items, publishes them, and issues the TMA loads
//   warp 9          owns tensor memory; issues every MMA (converged warp, one
//                   elected lane)
//   warp 10         cleans V tiles that not every row sees whole (below)
// Tensor memory (512 columns): S/P of A [0,128), of B [128,256), O of A
// [256,256+D), O of B [256+D,256+2D).  Per key tile the MMA warp issues P V and,
// once that product has read P (same columns), the next Q K^T, for A and B in
// turn: one side's products run while the other's softmax does.
//
// Softmax: a row's 128 scores are read from tensor memory into registers in one
// go; online, in base 2, with a running max that is raised, and O rescaled,
// only when it grows by more than 2^8 (fp16: 2^4, below).
//
// Large scores: a weight is 2^(s * scale_log2 - max) in one fused step, whose
// product is not rounded while the max's was.  All weights of a row share the
// difference, half a step of the max, and it cancels, unless it is so large that
// weights overflow or vanish.  From a max on whose step is worth several times a
// weight (kWide), the factor is the power of two above scale_log2, whose products
// are exact: a key with the row's largest score has weight 1, and one of the next
// score that fp32 knows, a step below, weighs less than the largest's rounding
// left open.  (The scores' distance from their max, taken first, is exact too but
// made prompts 6% slower: 160 -> 169 us, 770 -> 815 us.)
//
// Probabilities enter P.V as one 16-bit value when the output is 16 bits wide
// (each is off by half a step at most, the size of the output's own
// rounding), and as hi + lo 16-bit parts, two products, when it is fp32.
// Sums are taken of the fp32 probabilities.  Two parts for 16-bit outputs would
// bring the error against 64 bits from 1.1-1.4 times the final rounding's down
// to it, for a longer chain: 1641 rows 30.7 -> 42.1 us on the device, ragged
// prompts 154 -> 218, 8192 rows 731 -> 1079, long trees 201 -> 271.
//
// 0 x NaN: a masked key has probability 0, but its V may hold anything.  In a
// key tile that is not seen whole by every row, V rows that no row sees are
// zeroed in shared memory, and NaNs and infinities of the others too; rows
// that do see such a value get it back in the epilogue (a rare path that
// reads V again, and that also undoes infinity x 0 where a part of P is 0).
#include "pa_device.h"
#include "pa_prompt_plan.cuh"
#include "pa_ptx.cuh"
#include "pa_serving.h"
#include "pa_tc.cuh"
#include "pa_tree_plan.cuh"

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace pa {

namespace {

constexpr int kBM = 128;  // MMA rows of a row tile
constexpr int kBN = 128;  // keys of a tile
constexpr int kKS = 3;    // K ring depth
constexpr int kVS = 2;    // V ring depth
constexpr int kIS = 2;    // items published ahead
constexpr int kAsk = 8;   // CTAs that one past the last unit cancels at a time
constexpr int kThreads = 384;  // three warpgroups
// registers of a thread: 2 x 184 + 128 of the launch's 3 x 168 (208 + 88 was slower: the others spilled)
constexpr int kSoftmaxRegs = 184, kOtherRegs = 128;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kCleanWarp = 10;
constexpr uint32_t kHalfBytes = kBN * 128;  // one 64-dim half of a tile
constexpr uint64_t kWaitNs = 2000000000ull;  // a role gives up after 2 s on one barrier
constexpr uint32_t kSleepNs = 20000;        // longest sleep inside one try_wait
constexpr int kWaitSlices = int(kWaitNs / kSleepNs);
// What a tree's unit costs apart from its key tiles, in key tiles of a twin
// (0.9 us each; 1.75 us with two row tiles): start, joins and epilogue, 4.5 us
constexpr int kUnitStart = 5;
constexpr uint32_t kNegInf = 0xff800000u, kPosInf = 0x7f800000u, kNan = 0x7fffffffu;

struct Item {
    TreeItem t;
    int valid;
};

struct Bars {
    uint64_t q_full, q_empty;
    uint64_t k_full[kKS], k_empty[kKS], v_full[kVS], v_clean[kVS], v_empty[kVS];
    uint64_t s_full[2], p_full[2], o_done[2];  // of row tile x
    uint64_t item_full[kIS], item_empty[kIS];
    uint64_t unit_asked;      // prompt: the units' numbers asked for have arrived
    alignas(16) uint4 unit[kAsk];
    uint64_t side_b, side_w;  // twin: `side` holds B's figures; the weights
    uint64_t twin_read;       // twin: side B has read A's O
    uint64_t mma_done, never;
    uint32_t tmem, abort;
    uint32_t poison[kIS];  // n + 1: item n met a NaN or infinity in a V that not every row sees
    Item items[kIS];
    float2 side[kBM];  // twin: B's max and sum, then both sides' weights, of each row
};

template <int D> struct Smem {
    static constexpr uint32_t kTileBytes = kBN * D * 2;  // one K (or V, or Q) tile
    static constexpr uint32_t kKOff = 2 * kTileBytes;    // after Q of A and B
    static constexpr uint32_t kVOff = kKOff + kKS * kTileBytes;
    static constexpr uint32_t kBarOff = kVOff + kVS * kTileBytes;
    static constexpr uint32_t kBytes = 1024 + kBarOff + sizeof(Bars);
};
static_assert(Smem<128>::kBytes <= 232448, "shared memory of one CTA");

__device__ inline uint32_t col_s(int x) { return 128u * x; }
template <int D> __device__ inline uint32_t col_o(int x) { return 256u + uint32_t(D) * x; }

struct TcArgs {
    PackedAttn a;
    TreeShape shape;
    PromptShape prompt;
    int32_t tq, G, head_first;
};

// Waits for a phase: one suspended try, then others of up to kSleepNs each, a
// bounded number of them, until another role has given up.  Kept short: every
// wait is a copy of this, and the SM's instruction cache is small.
__device__ inline bool wait_bar(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
    for (int i = 0; i < kWaitSlices; ++i) {
        if (mbar_try_wait_sleep(bar, parity, kSleepNs)) return true;
        if (*abort_flag) return false;
    }
    return false;
}

// MMA and commit by the lane for which `e` is 1, chosen once: an election inside
// each MMA made a product of eight 3.8 KB of code and the MMA warp's pace the
// kernel's (8192 rows, 64/8 heads, on one box: 744 against 714 us).
__device__ inline uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
    return r;
}
__device__ inline void mma_ss1(uint32_t d, uint64_t a, uint64_t b, uint32_t i, bool acc, uint32_t e) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(i), "r"(acc ? 1u : 0u), "r"(e) : "memory");
}
__device__ inline void mma_ts1(uint32_t d, uint32_t a, uint64_t b, uint32_t i, bool acc, uint32_t e) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(i), "r"(acc ? 1u : 0u), "r"(e) : "memory");
}
__device__ inline void commit1(uint64_t* bar, uint32_t e) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(e) : "memory");
}

__device__ inline float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Pairs of fp32 in one 64-bit register pair, and their paired arithmetic.
__device__ inline uint64_t f2_pack(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ inline void f2_unpack(uint64_t v, uint32_t& lo, uint32_t& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
__device__ inline uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ inline uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ inline uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ inline uint64_t f2_sub(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The 16-bit type's packing of two fp32 (low half = first), its exact halves
// back, and a test for NaNs and infinities: x * 0 is NaN for those alone.
template <typename T> struct H2;
template <> struct H2<__nv_bfloat16> {
    __device__ static inline uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static inline uint64_t unpack(uint32_t h) { return f2_pack(h << 16, h & 0xffff0000u); }
    __device__ static inline uint32_t probe(uint32_t x, uint32_t acc) {
        const __nv_bfloat162 z = __float2bfloat162_rn(0.f);
        const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), z,
                                         *reinterpret_cast<const __nv_bfloat162*>(&acc));
        return *reinterpret_cast<const uint32_t*>(&y);
    }
    static constexpr uint32_t kExp = 0x7f80u;
    static constexpr float kWide = 268435456.f;  // 2^28: below it half a step is 8 of exponent at most
    static constexpr float kShift = 0.f, kStep = 8.f;
};
template <> struct H2<__half> {
    __device__ static inline uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static inline uint64_t unpack(uint32_t h) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        return f2_pack(__float_as_uint(f.x), __float_as_uint(f.y));
    }
    __device__ static inline uint32_t probe(uint32_t x, uint32_t acc) {
        const __half2 z = __float2half2_rn(0.f);
        const __half2 y =
            __hfma2(*reinterpret_cast<const __half2*>(&x), z, *reinterpret_cast<const __half2*>(&acc));
        return *reinterpret_cast<const uint32_t*>(&y);
    }
    static constexpr uint32_t kExp = 0x7c00u;
    static constexpr float kWide = 16777216.f;  // 2^24: below it half a step is 1/2 of exponent at most
    // Weights below 2^-25, half of the least subnormal, are 0 in P but not in the
    // sum: were the max's weight 1, a history of 2^20 tokens just below would lose
    // 3% of a row.  It is 2^10 here and grows to 2^14 before the max is raised (2^15.5
    // with what rounding adds, of 65504): what a key loses is 2^-35 of the max's
    // weight at most.  (2^12, raised from 2^14 on, raised it too often: 34.2 us a
    // prompt of 1641 rows instead of 32.7.)
    static constexpr float kShift = 10.f, kStep = 4.f;
};
template <typename T> __device__ inline bool bad16(uint32_t h) { return (h & H2<T>::kExp) == H2<T>::kExp; }

__device__ inline uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

__device__ inline void apply_mask(uint32_t (&r)[32], uint32_t m) {
#pragma unroll
    for (int k = 0; k < 32; ++k) r[k] = ((m >> k) & 1u) ? r[k] : kNegInf;
}

__device__ inline float max32(const uint32_t (&r)[32]) {
    float m0 = __uint_as_float(r[0]), m1 = __uint_as_float(r[1]);
#pragma unroll
    for (int k = 2; k < 30; k += 4) {
        m0 = max3(m0, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
        m1 = max3(m1, __uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]));
    }
    return max3(fmaxf(m0, m1), __uint_as_float(r[30]), __uint_as_float(r[31]));
}

// A warp's 32 rows x kN 16-byte pieces, a row a lane, written so that four lanes
// write 64 consecutive bytes of a row: a store of a piece a lane touches 32
// lines and takes as long as four of these.  In groups of four lanes, lane b
// gets piece b of each of the group's rows (two rounds of exchanges).
// row(i) is the address of the group's i-th row, or nullptr where it is none.
template <int kN, typename Row> __device__ inline void store_rows4(uint4 (&v)[kN], int lane, Row row) {
    const bool up1 = lane & 1, up2 = lane & 2;
    auto swap = [&](uint4& a, uint4& b, bool up, int mask) {  // gives a (up) or b, takes the partner's
        uint4 x = up ? a : b;
        x.x = __shfl_xor_sync(0xffffffffu, x.x, mask);
        x.y = __shfl_xor_sync(0xffffffffu, x.y, mask);
        x.z = __shfl_xor_sync(0xffffffffu, x.z, mask);
        x.w = __shfl_xor_sync(0xffffffffu, x.w, mask);
        if (up)
            a = x;
        else
            b = x;
    };
#pragma unroll
    for (int g = 0; g < kN; g += 4) {
        swap(v[g], v[g + 1], up1, 1);
        swap(v[g + 2], v[g + 3], up1, 1);
        swap(v[g], v[g + 2], up2, 2);
        swap(v[g + 1], v[g + 3], up2, 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4* at = row(i);
            if (at) at[g + (lane & 3)] = v[g + i];
        }
    }
}

// What the two sides of an item do: their rows and key tiles.  Tile i of side x
// is the item's tile i, or 2 i + x of a twin, whose sides share A's rows.
struct Sides {
    int rows[2], tiles[2], nt;
    bool twin;
    __device__ inline int tile(int x, int i) const { return twin ? 2 * i + x : i; }
};
template <bool kTree> __device__ inline Sides sides_of(const TreeItem& t, int tq) {
    Sides s;
    s.nt = t.b1 - t.b0;
    s.rows[0] = min(tq, t.n_rows);
    s.rows[1] = t.n_rows - s.rows[0];
    s.twin = s.rows[1] == 0 && s.nt > 1;
    if (s.twin) {
        s.rows[1] = s.rows[0];
        s.tiles[0] = (s.nt + 1) >> 1;
        s.tiles[1] = s.nt >> 1;
    } else {  // causal: tile B may see one key tile more than A
        s.tiles[0] = kTree ? s.nt : (t.t0 + s.rows[0] + kBN - 1) / kBN;
        s.tiles[1] = s.rows[1] > 0 ? s.nt : 0;
    }
    return s;
}

// A prompt's grid has a CTA for each unit's number there can be; an SM holds one,
// and a CTA that is done asks the hardware to cancel the launch of a waiting one
// and takes its number, so that the longest units come first and none waits for
// a CTA that drew longer ones (numbers dealt out in turn instead: the ragged
// batch's CTAs ended between 95 and 180 us).
//
// Asks for the numbers of n CTAs that have not been launched; the answers (16
// bytes each) arrive on `bar`.  Not to be asked again after a refusal.
__device__ inline void ask_units(uint4* answer, int n, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, 16 * n);
#pragma unroll 1
    for (int i = 0; i < n; ++i) asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_u32(answer + i)),
        "r"(smem_u32(bar))
        : "memory");
}
// The number, or -1 for a refusal.
__device__ inline int answered_unit(uint4* answer) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    fence_proxy_async_smem();  // read before the next answer is written there
    return got ? int(x) : -1;
}

template <int N> __device__ inline void regs_grow() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ inline void regs_shrink() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <typename T, int D, bool kTree, typename TOut>
__global__ void __launch_bounds__(kThreads, 1)
    packed_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKc,
              const __grid_constant__ CUtensorMap tmVc, const __grid_constant__ TcArgs p) {
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr bool kSplit = std::is_same<TOut, float>::value;
    constexpr int kHalves = D / 64;  // 64-dim (128-byte) halves of a row
    constexpr uint32_t kTileBytes = Smem<D>::kTileBytes;
    const PackedAttn& a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.G, tq = p.tq;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* base =
        reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = base;
    Bars& B = *reinterpret_cast<Bars*>(base + Smem<D>::kBarOff);
    volatile uint32_t* abort_flag = &B.abort;
    auto k_tile = [&](int st) { return base + Smem<D>::kKOff + st * kTileBytes; };
    auto v_tile = [&](int st) { return base + Smem<D>::kVOff + st * kTileBytes; };

    if (tid == 0) {
        mbar_init(&B.q_full, 1);
        mbar_init(&B.q_empty, 1);
        for (int i = 0; i < kKS; ++i) {
            mbar_init(&B.k_full[i], 1);
            mbar_init(&B.k_empty[i], 1);
        }
        for (int i = 0; i < kVS; ++i) {
            mbar_init(&B.v_full[i], 1);
            mbar_init(&B.v_clean[i], 1);
            mbar_init(&B.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.s_full[i], 1);
            mbar_init(&B.p_full[i], 4);
            mbar_init(&B.o_done[i], 1);
        }
        for (int i = 0; i < kIS; ++i) {
            mbar_init(&B.item_full[i], 1);
            mbar_init(&B.item_empty[i], 10);  // 8 softmax warps, the MMA warp, the V warp
            B.poison[i] = 0;
        }
        mbar_init(&B.unit_asked, 1);
        mbar_init(&B.side_b, 4);
        mbar_init(&B.side_w, 4);
        mbar_init(&B.twin_read, 4);
        mbar_init(&B.mma_done, 1);
        mbar_init(&B.never, 1);
        B.abort = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&B.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = B.tmem;
    pdl_wait_primary();
    pdl_launch_dependents();  // after the wait, so that nothing overtakes what it waited for
    if (a.debug_timeout) {
        // Testing: a wait that runs out before any copy is issued (a barrier
        // nothing targets, no time allowed) aborts every role of the CTA.
        if (tid == 0 && !mbar_wait_ns(&B.never, 0, 0)) {
            *abort_flag = 1u;
            flag(a.dev_status, PA_DEV_TIMEOUT);
        }
        __syncthreads();
    }
    auto give_up = [&]() {
        *abort_flag = 1u;
        flag(a.dev_status, PA_DEV_TIMEOUT);
    };
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
    };
    if (warp == kProducerWarp) {
        // ================================ producer ================================
        regs_shrink<kOtherRegs>();
        if (lane == 0) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            if (kTree) {
                tma_prefetch_desc(&tmKc);
                tma_prefetch_desc(&tmVc);
            }
        }
        TreeWalk walk;
        PromptUnits units;
        if constexpr (kTree) {
            if (blockIdx.x == 0)
#pragma unroll 1
                for (int s = lane; s < p.shape.num_seqs; s += 32) {
                    const TreeSeq q = tree_seq(p.shape, s);
                    if (q.bad_rows || q.bad_len) flag(a.dev_status, PA_DEV_BAD_LEN);
                }
            walk.start(p.shape, blockIdx.x);
        } else {
            if (blockIdx.x == 0)
#pragma unroll 1
                for (int s = lane; s < a.r.num_seqs; s += 32) {
                    const int r0 = a.r.cu_lens[s], r1 = a.r.cu_lens[s + 1];
                    if (r0 < 0 || r1 < r0 || r1 > a.r.total_rows || r1 - r0 > a.r.max_rows)
                        flag(a.dev_status, PA_DEV_BAD_LEN);
                }
            units.start(p.prompt);
        }
        const int P = a.c.page_size;
        const int xc_first = p.head_first;
        int kq = 0, vq = 0, qn = 0;  // K tiles, V tiles and Qs issued
        int asks = 0, batch = 1;     // times that numbers were asked for, how many last
        int number = lane == 0 ? int(blockIdx.x) : -1;  // units' numbers at hand, one a lane
        bool ok = !*abort_flag, asked = false, refused = false, joins = false;
#pragma unroll 1
        for (int n = 0; ok; ++n) {
            Item it;
            if constexpr (kTree) {
                it.valid = walk.next(p.shape, it.t);
                if (it.valid ? begins(it.t) : !joins) {  // what there is to join here, or that there is nothing
                    if (lane == 0)
                        tree_joins(a.workspace, 2 * kBM, D, a.n_ctas)[blockIdx.x] =
                            it.valid ? join_of(it.t) : make_int4(0, 0, 0, 0);
                    joins = true;
                }
            } else {
                // A CTA whose number is past the last unit cancels those that wait, as
                // they are past it too, until there are none: quicker than their launch
                // (one prompt of 100 rows, 64/8 heads, replayed on a graph of 32768: 100
                // us with each launched, 22 us so).
                it.valid = 0;
#pragma unroll 1
                while (ok) {
                    const unsigned m = __ballot_sync(0xffffffffu, number >= 0);
                    if (m) {
                        const int l = __ffs(m) - 1, i = __shfl_sync(0xffffffffu, number, l);
                        if (lane == l) number = -1;
                        it.valid = units.get(p.prompt, i, it.t);
                        if (it.valid) break;
                    } else if (refused) {
                        break;
                    } else {
                        if (!asked) {  // else before the last item's last tile
                            batch = kAsk;
                            if (lane == 0) ask_units(B.unit, batch, &B.unit_asked);
                            ++asks;
                            asked = true;
                        }
                        ok = wait_all(&B.unit_asked, (asks - 1) & 1);
                        if (!ok) break;
                        asked = false;
                        if (lane < batch) number = answered_unit(&B.unit[lane]);
                        refused = __any_sync(0xffffffffu, lane < batch && number < 0);
                    }
                }
                if (!ok) break;
            }
            const int is = n % kIS;
            if (n >= kIS) ok = wait_all(&B.item_empty[is], ((n / kIS) - 1) & 1);
            if (!ok) break;
            if (lane == 0) {
                B.items[is] = it;
                mbar_arrive(&B.item_full[is]);
            }
            if (!it.valid) break;
            const TreeItem& t = it.t;
            const Sides sd = sides_of<kTree>(t, tq);
            const int nt = sd.nt, n_q = t.n_rows > tq ? 2 : 1;  // row tiles
            const int32_t* table = kTree ? a.c.block_tables + int64_t(t.seq) * a.c.max_blocks : nullptr;
            const int PT = kTree ? kBN / P : 0;
            const int npg = kTree ? (t.L + P - 1) / P : 0;
#pragma unroll 1
            for (int j = 0; j < nt; ++j) {
                if (!kTree && j == nt - 1) {
                    // unless there are numbers at hand or none left (a warp-wide test)
                    if (!refused && !__any_sync(0xffffffffu, number >= 0)) {
                        batch = 1;
                        if (lane == 0) ask_units(B.unit, batch, &B.unit_asked);
                        ++asks;
                        asked = true;
                    }
                }
                const int blk = t.b0 + j;
                const bool hist = kTree && blk < t.nh;
                int pg = a.c.num_pages;  // beyond the tensor: the box reads as zeros
                if (hist) {
                    const int idx = blk * PT + lane;
                    if (lane < PT && idx < npg) {
                        const int e = table[idx];
                        if (e >= 0 && e < a.c.num_pages)
                            pg = e;
                        else
                            flag(a.dev_status, PA_DEV_BAD_PAGE);
                    }
                }
                const int prow = t.row0 - t.t0 + (blk - t.nh) * kBN;  // packed row of the tile's first key
                auto load = [&](uint8_t* dst, const CUtensorMap* packed, const CUtensorMap* paged, uint64_t* bar) {
                    if (lane == 0) mbar_arrive_expect_tx(bar, kTileBytes);  // zero-filled boxes count whole
                    __syncwarp();
                    if (hist) {
                        if (lane < PT)
#pragma unroll
                            for (int hh = 0; hh < kHalves; ++hh)
                                tma_load_4d(dst + hh * kHalfBytes + lane * P * 128, paged, bar, 64 * hh,
                                            xc_first ? t.g : 0, xc_first ? 0 : t.g, pg);
                    } else if (lane < kHalves) {
                        tma_load_3d(dst + lane * kHalfBytes, packed, bar, 64 * lane, t.g, prow);
                    }
                };
                const int sk = kq % kKS, sv = vq % kVS;
                if (kq >= kKS) ok = wait_all(&B.k_empty[sk], ((kq / kKS) - 1) & 1);
                if (!ok) break;
                load(k_tile(sk), &tmK, &tmKc, &B.k_full[sk]);
                ++kq;
                if (j == 0) {
                    // Q, after the item's first K tile: the last item's products may still read its place
                    if (n > 0) ok = wait_all(&B.q_empty, (n - 1) & 1);
                    if (!ok) break;
                    if (lane == 0) {
                        const uint32_t qbytes = uint32_t(kHalves) * 128u * uint32_t(G * tq);
                        mbar_arrive_expect_tx(&B.q_full, n_q * qbytes);
                        for (int x = 0; x < n_q; ++x)
                            for (int hh = 0; hh < kHalves; ++hh)
                                tma_load_3d(sQ + x * kTileBytes + hh * kHalfBytes, &tmQ, &B.q_full, 64 * hh,
                                            t.g * G, t.row0 + x * tq);
                    }
                    ++qn;
                }
                if (vq >= kVS) ok = wait_all(&B.v_empty[sv], ((vq / kVS) - 1) & 1);
                if (!ok) break;
                load(v_tile(sv), &tmV, &tmVc, &B.v_full[sv]);
                ++vq;
            }
        }
        if (lane == 0) {
            if (kTree && !joins)  // gave up
                tree_joins(a.workspace, 2 * kBM, D, a.n_ctas)[blockIdx.x] = make_int4(0, 0, 0, 0);
            if (!ok) give_up();
            // never leave the CTA with copies in flight
            if (asked) mbar_wait_ns(&B.unit_asked, (asks - 1) & 1, kWaitNs);
#pragma unroll 1
            for (int j = max(0, kq - kKS); j < kq; ++j) mbar_wait_ns(&B.k_full[j % kKS], (j / kKS) & 1, kWaitNs);
#pragma unroll 1
            for (int j = max(0, vq - kVS); j < vq; ++j) mbar_wait_ns(&B.v_full[j % kVS], (j / kVS) & 1, kWaitNs);
            if (qn > 0 && !mbar_wait_ns(&B.q_full, (qn - 1) & 1, kWaitNs)) flag(a.dev_status, PA_DEV_TIMEOUT);
        }
    } else if (warp == kMmaWarp) {
        // ================================== MMA ===================================
        regs_shrink<kOtherRegs>();
        const uint32_t el = elect_one();
        const uint32_t idQK = tc::idesc_f16(kBM, kBN, kBf16, false);
        const uint32_t idPV = tc::idesc_f16(kBM, D, kBf16, true);
        // descriptors: the high word is shared, low words advance by offset >> 4
        const uint32_t hi_d = tc::desc_hi_sw128(1024);
        const uint32_t q_lo = tc::desc_lo(smem_u32(sQ), 16);
        const uint32_t k_lo = tc::desc_lo(smem_u32(k_tile(0)), 16);
        const uint32_t v_lo = tc::desc_lo(smem_u32(v_tile(0)), kHalfBytes);
        // S_x = Q K^T of row tile qt and K tile number t
        auto qk = [&](int x, int qt, int t) {
            const uint32_t qx = q_lo + qt * (kTileBytes >> 4);
            const uint32_t kx = k_lo + (t % kKS) * (kTileBytes >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
                mma_ss1(tm + col_s(x), tc::make_desc(qx + off, hi_d), tc::make_desc(kx + off, hi_d), idQK, ks > 0, el);
            }
            commit1(&B.s_full[x], el);
        };
        // O_x (+)= P_x V of V tile number t.  16 keys: 8 columns of P, 2048 bytes
        // of V; P of 32 keys takes 16 columns (kSplit: 32, hi then lo, a product each)
        auto pv = [&](int x, int t, bool first) {
            const uint32_t vx = v_lo + (t % kVS) * (kTileBytes >> 4);
            const uint32_t p_col = tm + col_s(x), o_col = tm + col_o<D>(x);
#pragma unroll
            for (int ks = 0; ks < kBN / 16; ++ks) {
                const uint64_t bd = tc::make_desc(vx + ks * (2048 >> 4), hi_d);
                if constexpr (kSplit) {
                    const uint32_t col = p_col + 32 * (ks >> 1) + 8 * (ks & 1);
                    mma_ts1(o_col, col, bd, idPV, !first || ks > 0, el);
                    mma_ts1(o_col, col + 16, bd, idPV, true, el);
                } else {
                    mma_ts1(o_col, p_col + 8 * ks, bd, idPV, !first || ks > 0, el);
                }
            }
            commit1(&B.o_done[x], el);
        };
        auto have_k = [&](int t) { return wait_all(&B.k_full[t % kKS], (t / kKS) & 1); };
        auto have_v = [&](int t) { return wait_all(&B.v_clean[t % kVS], (t / kVS) & 1); };
        int kt = 0;          // K and V tiles of the items before
        int sc[2] = {0, 0};  // score tiles of x issued; P_x V number sc - 1 waits for its P
        int twins = 0;       // twins before this item
        bool behind_twin = false;
        // P V of side x with tile t.  Behind it, where this warp would wait anyway,
        // stand the commits and the next tiles' waits.
        auto take_p = [&](int x, int t, bool first) {
            if (!wait_all(&B.p_full[x], (sc[x] - 1) & 1)) return false;
            // Side B of a twin reads A's O too, which A's P of the next item does not
            // wait for.  (A has read B's O by then: its P comes first in every item.)
            if (x == 0 && first && behind_twin && !wait_all(&B.twin_read, (twins - 1) & 1)) return false;
            tc::fence_after_sync();
            pv(x, t, first);
            return true;
        };
        // Q K^T of the side's next tile takes the place of its P (of the last
        // item's, at first): once that P V is done
        auto next_s = [&](int x, int qt, int t) {
            if (sc[x] > 0 && !wait_all(&B.o_done[x], (sc[x] - 1) & 1)) return false;
            tc::fence_after_sync();
            qk(x, qt, t);
            ++sc[x];
            return true;
        };
        auto run_twin = [&](int nt) {  // side x: tiles x, x + 2, ...
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (x == 1 && !have_k(kt + 1)) return false;
                if (!next_s(x, 0, kt + x)) return false;
                commit1(&B.k_empty[(kt + x) % kKS], el);
            }
            if (nt == 2) commit1(&B.q_empty, el);
            if (!have_v(kt)) return false;
#pragma unroll 1
            for (int j = 0; j < nt; j += 2) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int t = kt + j + x;
                    if (j + x >= nt) return true;
                    if (!take_p(x, t, j == 0)) return false;
                    commit1(&B.v_empty[t % kVS], el);
                    if (j + x + 1 < nt && !have_v(t + 1)) return false;
                    if (j + x + 2 < nt) {
                        if (!have_k(t + 2) || !next_s(x, 0, t + 2)) return false;
                        commit1(&B.k_empty[(t + 2) % kKS], el);
                        if (j + x + 3 == nt) commit1(&B.q_empty, el);
                    }
                }
            }
            return true;
        };
        auto run_pair = [&](const Sides& sd) {  // both sides take every tile (A alone, where there is no B)
            const int nt = sd.nt;
            const bool two = sd.tiles[1] > 0;
            if (!next_s(0, 0, kt) || (two && !next_s(1, 1, kt))) return false;
            commit1(&B.k_empty[kt % kKS], el);
            if (nt == 1) commit1(&B.q_empty, el);
            if (!have_v(kt)) return false;
#pragma unroll 1
            for (int j = 0; j < nt; ++j) {
                const int t = kt + j;
                const bool more = j + 1 < nt;
                if (j < sd.tiles[0] && !take_p(0, t, j == 0)) return false;
                if (more && !have_k(t + 1)) return false;
                if (j + 1 < sd.tiles[0] && !next_s(0, 0, t + 1)) return false;
                if (two && !take_p(1, t, j == 0)) return false;
                commit1(&B.v_empty[t % kVS], el);
                if (!more) return true;
                if (!have_v(t + 1) || (two && !next_s(1, 1, t + 1))) return false;
                commit1(&B.k_empty[(t + 1) % kKS], el);
                if (j + 2 == nt) commit1(&B.q_empty, el);
            }
            return true;
        };
        auto run = [&]() {
#pragma unroll 1
            for (int n = 0;; ++n) {
                const int is = n % kIS;
                if (!wait_all(&B.item_full[is], (n / kIS) & 1)) return false;
                const int valid = B.items[is].valid;
                const Sides sd = sides_of<kTree>(B.items[is].t, tq);
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.item_empty[is]);
                if (!valid) return true;
                if (!wait_all(&B.q_full, n & 1) || !have_k(kt)) return false;
                if (!(sd.twin ? run_twin(sd.nt) : run_pair(sd))) return false;
                behind_twin = sd.twin;
                twins += sd.twin;
                kt += sd.nt;
            }
        };
        if (!run() && lane == 0) give_up();
        // every MMA issued so far has finished before tensor memory is freed
        commit1(&B.mma_done, el);
        if (!__all_sync(0xffffffffu, mbar_wait_ns(&B.mma_done, 0, kWaitNs)) && lane == 0)
            flag(a.dev_status, PA_DEV_TIMEOUT);
    } else if (warp == kCleanWarp) {
        // ================================= V rows ==================================
        regs_shrink<kOtherRegs>();
        int vt = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            const int is = n % kIS;
            ok = wait_all(&B.item_full[is], (n / kIS) & 1);
            if (!ok || !B.items[is].valid) break;
            const TreeItem t = B.items[is].t;
#pragma unroll 1
            for (int j = 0; j < t.b1 - t.b0; ++j, ++vt) {
                const int blk = t.b0 + j, sv = vt % kVS;
                const bool hist = kTree && blk < t.nh;
                const int k0 = (blk - (hist ? 0 : t.nh)) * kBN;
                const int v_end = hist ? t.L : kTree ? t.T : t.t0 + t.n_rows;  // keys that some row sees
                const bool mixed = kTree ? !hist : k0 + kBN > t.t0 + 1;        // keys that only some rows see
                ok = wait_all(&B.v_full[sv], (vt / kVS) & 1);
                if (!ok) break;
                if (mixed || k0 + kBN > v_end) {
#pragma unroll 1
                    for (int r = lane; r < kBN; r += 32) {
                        uint8_t* row = v_tile(sv) + r * 128;  // a key's row, 64 dims at a time
                        if (k0 + r >= v_end) {
#pragma unroll
                            for (int c = 0; c < D / 8; ++c)
                                *reinterpret_cast<uint4*>(row + (c >> 3) * kHalfBytes + ((c + lane) & 7) * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        } else if (mixed) {
                            uint32_t acc = 0u;
#pragma unroll
                            for (int c = 0; c < D / 8; ++c) {
                                const uint4 w = *reinterpret_cast<const uint4*>(row + (c >> 3) * kHalfBytes +
                                                                                ((c + lane) & 7) * 16);
                                acc = H2<T>::probe(w.x, H2<T>::probe(w.y, H2<T>::probe(w.z, H2<T>::probe(w.w, acc))));
                            }
                            if (bad16<T>(acc) || bad16<T>(acc >> 16)) {
#pragma unroll 1
                                for (int c = 0; c < D / 2; ++c) {
                                    uint32_t* w = reinterpret_cast<uint32_t*>(row + (c >> 5) * kHalfBytes) + (c & 31);
                                    uint32_t y = *w;
                                    if (bad16<T>(y)) y &= 0xffff0000u;
                                    if (bad16<T>(y >> 16)) y &= 0x0000ffffu;
                                    *w = y;
                                }
                                B.poison[is] = uint32_t(n) + 1u;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.v_clean[sv]);
            }
            if (ok && lane == 0) mbar_arrive(&B.item_empty[is]);
        }
        if (!ok && lane == 0) give_up();
    } else if (warp > kCleanWarp) {
        regs_shrink<kOtherRegs>();  // an idle warp: the whole warpgroup gives
    } else {
        // ================================= softmax =================================
        regs_grow<kSoftmaxRegs>();
        const int x = warp >> 2;  // side
        const int quad = warp & 3;
        const int m = quad * 32 + lane;  // MMA row = tensor-memory lane
        const uint32_t lane_addr = uint32_t(quad * 32) << 16;
        const int tr = m / G, h = m - tr * G;
        const float sl2 = a.scale_log2;
        const float sl2_wide = __uint_as_float((__float_as_uint(sl2) + 0x007fffffu) & 0x7f800000u);
        const uint32_t sbase = tm + lane_addr + col_s(x);
        const uint32_t obase = tm + lane_addr + col_o<D>(x);
        int sc = 0, sc_other = 0;  // score tiles of this side and of the other before this item
        int twins = 0;             // twins before it
        bool ok = true;
        for (int n = 0; ok; ++n) {
            const int is = n % kIS;
            ok = wait_all(&B.item_full[is], (n / kIS) & 1);
            if (!ok) break;
            const TreeItem t = B.items[is].t;
            if (!B.items[is].valid) break;
            const Sides sd = sides_of<kTree>(t, tq);
            const int nt = x ? sd.tiles[1] : sd.tiles[0];
            const bool row_ok = tr < tq && tr < (x ? sd.rows[1] : sd.rows[0]);
            const int tile_row = (sd.twin ? 0 : x * tq) + tr;
            const int tt = t.t0 + tile_row;  // the row's place in its sequence
            const int row = t.row0 + tile_row;
            const int P = a.c.page_size;
            const int32_t* table = kTree ? a.c.block_tables + int64_t(t.seq) * a.c.max_blocks : nullptr;
            const int PT = kTree ? kBN / P : 0;
            const int npg = kTree ? (t.L + P - 1) / P : 0;
            // table entry of page `lane` of a history tile (0, a page inside the pool, past its pages)
            auto entry = [&](int blk) -> int {
                const int idx = blk * PT + lane;
                return kTree && blk < t.nh && lane < PT && idx < npg ? __ldg(table + idx) : 0;
            };
            float m_run = -INFINITY, l_run = 0.f;
            int e_cur = entry(t.b0 + sd.tile(x, 0));
#pragma unroll 1
            for (int i = 0; i < nt; ++i) {
                const int blk = t.b0 + sd.tile(x, i);
                const bool hist = kTree && blk < t.nh;
                const int k0 = (blk - (hist ? 0 : t.nh)) * kBN;  // first key, of the history or the packed rows
                const int e_nxt = kTree && i + 1 < nt ? entry(t.b0 + sd.tile(x, i + 1)) : 0;
                uint32_t see[4];  // keys of this tile that the row sees
                if (hist) {
                    const uint32_t pmask = __ballot_sync(0xffffffffu, e_cur >= 0 && e_cur < a.c.num_pages);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        see[c] = low_bits(t.L - k0 - 32 * c);
                        if (P == 32)
                            see[c] &= (pmask >> c) & 1u ? 0xffffffffu : 0u;
                        else
                            see[c] &= ((pmask >> (2 * c)) & 1u ? 0x0000ffffu : 0u) |
                                      ((pmask >> (2 * c + 1)) & 1u ? 0xffff0000u : 0u);
                    }
                } else if constexpr (kTree) {
                    const uint32_t* words = a.tree_mask + int64_t(row) * a.mask_words + (k0 >> 5);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        see[c] = row_ok && !t.bad_len && (k0 >> 5) + c < a.mask_words
                                     ? __ldg(words + c) & low_bits(t.T - k0 - 32 * c)
                                     : 0u;
                } else {
                    const int lim = row_ok ? tt + 1 - k0 : 0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) see[c] = low_bits(lim - 32 * c);
                }
                e_cur = e_nxt;
                ok = wait_all(&B.s_full[x], (sc + i) & 1);
                if (!ok) break;
                tc::fence_after_sync();

                // ---- p = 2^(s * scale_log2 - m_run) of the row's 128 scores
                uint32_t r[4][32];
                float sum;
                {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::ld_32x32b_x32(sbase + 32 * c, r[c]);
                    tc::wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tc::reg_fence(r[c]);
                        if (see[c] != 0xffffffffu) apply_mask(r[c], see[c]);
                    }
                    float mx[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) mx[c] = max32(r[c]);
                    const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                    const float low = top * sl2 - H2<T>::kShift;
                    const float mt = fabsf(low) < H2<T>::kWide ? low : top * sl2_wide;
                    const bool need = mt - m_run > H2<T>::kStep;  // false for two infinities of a sign
                    // raise the max and rescale O in place: the last P V has
                    // finished (these scores were issued after it)
                    const float alpha = need ? ex2(m_run - mt) : 1.f;
                    if (need) m_run = mt;
                    l_run *= alpha;
                    if (i > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t ro[16];
                            tc::ld_32x32b_x16(obase + 16 * c, ro);
                            tc::wait_ld();
                            tc::reg_fence(ro);
#pragma unroll
                            for (int k = 0; k < 16; ++k) ro[k] = __float_as_uint(__uint_as_float(ro[k]) * alpha);
                            tc::st_32x32b_x16(obase + 16 * c, ro);
                        }
                    }
                    const float nmu = m_run == -INFINITY ? 0.f : -m_run;  // nothing seen yet: weights 0, not NaN
                    const float f = fabsf(nmu) < H2<T>::kWide ? sl2 : sl2_wide;
                    const uint64_t sl2_2 = f2_pack(__float_as_uint(f), __float_as_uint(f));
                    const uint64_t nmu_2 = f2_pack(__float_as_uint(nmu), __float_as_uint(nmu));
                    uint64_t sum_2[2] = {f2_pack(0u, 0u), f2_pack(0u, 0u)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
#pragma unroll
                        for (int w = 0; w < 16; ++w) {
                            uint32_t z0, z1;
                            f2_unpack(f2_fma(f2_pack(r[c][2 * w], r[c][2 * w + 1]), sl2_2, nmu_2), z0, z1);
                            const float p0 = ex2(__uint_as_float(z0)), p1 = ex2(__uint_as_float(z1));
                            const uint64_t pp = f2_pack(__float_as_uint(p0), __float_as_uint(p1));
                            sum_2[w & 1] = f2_add(sum_2[w & 1], pp);
                            r[c][2 * w] = H2<T>::pack(p0, p1);
                            if constexpr (kSplit) {
                                uint32_t d0, d1;
                                f2_unpack(f2_sub(pp, H2<T>::unpack(r[c][2 * w])), d0, d1);
                                r[c][2 * w + 1] = H2<T>::pack(__uint_as_float(d0), __uint_as_float(d1));
                            }
                        }
                    }
                    uint32_t s0, s1;
                    f2_unpack(f2_add(sum_2[0], sum_2[1]), s0, s1);
                    sum = __uint_as_float(s0) + __uint_as_float(s1);
                }
                l_run += sum;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if constexpr (kSplit) {
                        tc::st_32x32b_x16_stride2<0>(sbase + 32 * c, r[c]);
                        tc::st_32x32b_x16_stride2<1>(sbase + 32 * c + 16, r[c]);
                    } else {
                        tc::st_32x32b_x16_stride2<0>(sbase + 16 * c, r[c]);
                    }
                }
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.p_full[x]);
            }
            if (!ok) break;

            // Puts right 32 dims of the rows that `mine` marks, which may see a NaN or
            // infinity in V: one that was kept out of P.V, or that met a zero part
            // of P there.  What a row sees of them is the result, whatever the rest
            // adds up to.  The whole warp looks for them, a key a lane, and each row
            // keeps a bit for each kind and dim (20000 rows, 2/1 heads of 64, a NaN in
            // one of them: 0.45 ms, 0.21 ms without it, 45 ms when each row went
            // through its keys by itself; infinities in all: 3.1 ms, 47 ms when the
            // dims were added up one after another, at heads of 128 7.2 and 263).
            auto restore = [&](uint32_t (&r)[32], const TreeItem& it, int at, int place, int d0, bool mine) {
                uint32_t nan = 0u, pos = 0u, neg = 0u;  // what the row has seen: a bit a dim
                const int n_hist = kTree ? max(0, min(it.L, min(it.b1, it.nh) * kBN) - it.b0 * kBN) : 0;
                const int k_lo = max(0, it.b0 - it.nh) * kBN;
                const int k_hi = kTree ? min(it.T, max(0, it.b1 - it.nh) * kBN) : it.t0 + it.n_rows;
                const int n_keys = n_hist + max(0, k_hi - k_lo);
                bool left = mine;  // false once all that can follow changes nothing
#pragma unroll 1
                for (int i0 = 0; i0 < n_keys && __any_sync(0xffffffffu, left); i0 += 32) {
                    const int i = i0 + lane;
                    const T* v = nullptr;
                    if (kTree && i < n_hist) {
                        const int key = it.b0 * kBN + i, pg = table[key / P];
                        if (pg >= 0 && pg < a.c.num_pages)
                            v = static_cast<const T*>(a.c.v) + int64_t(pg) * a.c.page_stride +
                                int64_t(key % P) * a.c.token_stride + int64_t(it.g) * a.c.head_stride + d0;
                    } else if (i < n_keys) {
                        v = static_cast<const T*>(a.v) + int64_t(it.row0 - it.t0 + k_lo + i - n_hist) * a.r.v_stride +
                            it.g * D + d0;
                    }
                    uint32_t acc = 0u;
                    if (v) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 w = reinterpret_cast<const uint4*>(v)[c];
                            acc = H2<T>::probe(w.x, H2<T>::probe(w.y, H2<T>::probe(w.z, H2<T>::probe(w.w, acc))));
                        }
                    }
                    unsigned m = __ballot_sync(0xffffffffu, bad16<T>(acc) || bad16<T>(acc >> 16));
#pragma unroll 1
                    for (; m; m &= m - 1) {
                        const int l = __ffs(m) - 1, key = k_lo + i0 + l - n_hist;
                        const T* u = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(v), l));
                        bool sees = left;
                        if (i0 + l >= n_hist) {
                            if constexpr (kTree)
                                sees = sees && (key >> 5) < a.mask_words &&
                                       ((a.tree_mask[int64_t(at) * a.mask_words + (key >> 5)] >> (key & 31)) & 1u);
                            else
                                sees = sees && key <= place;
                        }
                        if (!__any_sync(0xffffffffu, sees)) continue;
                        const float y = Elt<T>::f(u[lane]);  // a dim a lane
                        const uint32_t yn = __ballot_sync(0xffffffffu, y != y);
                        const uint32_t yp = __ballot_sync(0xffffffffu, y == INFINITY);
                        const uint32_t ym = __ballot_sync(0xffffffffu, y == -INFINITY);
                        if (sees) {
                            pos |= yp;
                            neg |= ym;
                            nan |= yn | (pos & neg);
                            left = nan != 0xffffffffu;
                        }
                    }
                }
                if (!mine) return;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    if ((pos >> k) & 1u) r[k] = kPosInf;
                    if ((neg >> k) & 1u) r[k] = kNegInf;
                    if ((nan >> k) & 1u) r[k] = kNan;
                }
            };

            // ---- epilogue: O / l, or the piece's max, sum and O into its slot.  A
            // twin's rows are joined: each side writes half of the dims.
            sc += nt;
            sc_other += x ? sd.tiles[0] : sd.tiles[1];
            if (nt > 0) {
                ok = wait_all(&B.o_done[x], (sc - 1) & 1);
                if (ok && sd.twin) ok = wait_all(&B.o_done[1 - x], (sc_other - 1) & 1);
                if (!ok) break;
                tc::fence_after_sync();
                const bool poison = *reinterpret_cast<volatile uint32_t*>(&B.poison[is]) == uint32_t(n) + 1u;
                const bool piece = kTree && t.slot >= 0;
                float2 w = make_float2(1.f, 0.f);  // what side A's (or the only) O counts, and side B's
                if (sd.twin) {  // threads m of both sides hold the same row: B's figures, then A's verdict
                    if (x == 1) {
                        B.side[m] = make_float2(m_run, l_run);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&B.side_b);
                    } else {
                        ok = wait_all(&B.side_b, twins & 1);
                        if (!ok) break;
                        const float2 o = B.side[m];
                        const float top = fmaxf(m_run, o.x), base = top == -INFINITY ? 0.f : top;
                        w = make_float2(ex2(m_run - base), ex2(o.x - base));
                        // max drops NaN, so a sum may be NaN beside a max of -inf
                        l_run = (l_run == 0.f ? 0.f : l_run * (m_run == -INFINITY ? 1.f : w.x)) +
                                (o.y == 0.f ? 0.f : o.y * (o.x == -INFINITY ? 1.f : w.y));
                        m_run = top;
                    }
                }
                if (!piece && (x == 0 || !sd.twin)) {
                    const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
                    w.x *= inv;
                    w.y *= inv;
                }
                if (sd.twin) {
                    if (x == 0) {
                        B.side[m] = w;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&B.side_w);
                    } else {
                        ok = wait_all(&B.side_w, twins & 1);
                        if (!ok) break;
                        w = B.side[m];
                    }
                    ++twins;
                }
                const int r_unit = tile_row * G + h;  // distribution of the unit
                float* slot = piece ? static_cast<float*>(a.workspace) + slot_floats(2 * kBM, D) * t.slot : nullptr;
                TOut* orow = static_cast<TOut*>(a.out) + (int64_t(row) * a.Hq + t.g * G + h) * D;
                if (piece && row_ok && (x == 0 || !sd.twin))
                    *reinterpret_cast<float2*>(slot + 2 * r_unit) = make_float2(m_run, l_run);
                const int c_lo = sd.twin ? x * (D / 64) : 0, c_hi = sd.twin ? c_lo + D / 64 : D / 32;
#pragma unroll 1
                for (int c = c_lo; c < c_hi; ++c) {
                    uint32_t r[32];
                    tc::ld_32x32b_x32((sd.twin ? tm + lane_addr + col_o<D>(0) : obase) + 32 * c, r);
                    const uint64_t wx = f2_pack(__float_as_uint(w.x), __float_as_uint(w.x));
                    uint64_t z = 0;  // x * 0 is NaN for NaNs and infinities alone
                    if (sd.twin) {
                        uint32_t o[32];
                        tc::ld_32x32b_x32(tm + lane_addr + col_o<D>(1) + 32 * c, o);
                        tc::wait_ld();
                        tc::reg_fence(r);
                        tc::reg_fence(o);
                        const uint64_t wy = f2_pack(__float_as_uint(w.y), __float_as_uint(w.y));
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const uint64_t y = f2_fma(f2_pack(o[k], o[k + 1]), wy, f2_mul(f2_pack(r[k], r[k + 1]), wx));
                            f2_unpack(y, r[k], r[k + 1]);
                            z = f2_fma(y, 0ull, z);
                        }
                    } else {
                        tc::wait_ld();
                        tc::reg_fence(r);
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const uint64_t y = f2_mul(f2_pack(r[k], r[k + 1]), wx);
                            f2_unpack(y, r[k], r[k + 1]);
                            z = f2_fma(y, 0ull, z);
                        }
                    }
                    uint32_t z0, z1;
                    f2_unpack(z, z0, z1);
                    const float zz = __uint_as_float(z0) + __uint_as_float(z1);
                    const bool fix = row_ok && !t.bad_len && w.x == w.x && (poison || zz != zz);
                    if (__any_sync(0xffffffffu, fix)) restore(r, t, row, tt, 32 * c, fix);
                    __syncwarp();
                    // row i of this lane's group of four: its lane's own dst
                    auto row_at = [&](int i, uint64_t mine) {
                        return reinterpret_cast<uint4*>(__shfl_sync(0xffffffffu, mine, (lane & 28) + i));
                    };
                    if (piece || kSplit) {
                        const uint64_t mine = reinterpret_cast<uint64_t>(
                            !row_ok ? nullptr : (piece ? slot + 4 * kBM + int64_t(r_unit) * D : reinterpret_cast<float*>(orow)) + 32 * c);
                        uint4 y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
                        store_rows4(y, lane, [&](int i) { return row_at(i, mine); });
                    } else {
                        const uint64_t mine = reinterpret_cast<uint64_t>(row_ok ? orow + 32 * c : nullptr);
                        uint4 y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t* w4 = &y[k].x;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w4[e] = H2<T>::pack(__uint_as_float(r[8 * k + 2 * e]), __uint_as_float(r[8 * k + 2 * e + 1]));
                        }
                        store_rows4(y, lane, [&](int i) { return row_at(i, mine); });
                    }
                }
                if (sd.twin && x == 1) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B.twin_read);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.item_empty[is]);
        }
        if (!ok) give_up();
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tm, 512);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};  // the driver's, the same for every thread
    PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_relaxed);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
            known.store(fn, std::memory_order_relaxed);
        }
    }
    return fn;
}

bool encode(CUtensorMap* m, pa_dtype dt, int rank, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc && enc(m, dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                      const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed rows as (head_dim, head, row); the box is 64 dims x heads x rows.
bool encode_rows(CUtensorMap* m, const PackedAttn& a, const void* ptr, int heads, int64_t stride, int box_heads,
                 int box_rows) {
    const cuuint64_t dims[3] = {cuuint64_t(a.D), cuuint64_t(heads), cuuint64_t(a.r.total_rows)};
    const cuuint64_t strides[2] = {cuuint64_t(a.D) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)};
    return encode(m, a.dtype, 3, ptr, dims, strides, box);
}

// The pool as (head_dim, kv head, slot, page), the middle two in stride order;
// the box is one page of one kv head, 64 dims at a time.
bool encode_pages(CUtensorMap* m, const PackedAttn& a, const void* ptr, bool head_first) {
    const CacheArgs& c = a.c;
    const cuuint64_t hs = cuuint64_t(c.head_stride) * 2, ts = cuuint64_t(c.token_stride) * 2;
    const cuuint64_t nh = cuuint64_t(a.Hkv), P = cuuint64_t(c.page_size);
    const cuuint64_t dims[4] = {cuuint64_t(a.D), head_first ? nh : P, head_first ? P : nh, cuuint64_t(c.num_pages)};
    const cuuint64_t strides[3] = {head_first ? hs : ts, head_first ? ts : hs, cuuint64_t(c.page_stride) * 2};
    const cuuint32_t box[4] = {64, head_first ? 1u : cuuint32_t(P), head_first ? cuuint32_t(P) : 1u, 1};
    return encode(m, a.dtype, 4, ptr, dims, strides, box);
}

template <typename T, int D, bool kTree, typename TOut>
cudaError_t launch_typed(const PackedAttn& a, cudaStream_t st) {
    auto kern = packed_tc<T, D, kTree, TOut>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kern), Smem<D>::kBytes, allowed);
    if (e != cudaSuccess) return e;
    TcArgs p = {};
    p.a = a;
    p.G = a.Hq / a.Hkv;
    p.tq = kBM / p.G;
    CUtensorMap mq, mk, mv, mkc, mvc;
    if (!encode_rows(&mq, a, a.q, a.Hq, a.r.q_stride, p.G, p.tq) ||
        !encode_rows(&mk, a, a.k, a.Hkv, a.r.k_stride, 1, kBN) ||
        !encode_rows(&mv, a, a.v, a.Hkv, a.r.v_stride, 1, kBN))
        return cudaErrorInvalidValue;
    mkc = mk;
    mvc = mv;
    int64_t ctas;
    if (kTree) {
        p.head_first = a.c.head_stride <= a.c.token_stride;
        if (!encode_pages(&mkc, a, a.c.k, p.head_first) || !encode_pages(&mvc, a, a.c.v, p.head_first))
            return cudaErrorInvalidValue;
        TreeShape& s = p.shape;
        s.cu_lens = a.r.cu_lens;
        s.context_lens = a.c.context_lens;
        s.num_seqs = a.r.num_seqs;
        s.total_rows = a.r.total_rows;
        s.max_rows = a.r.max_rows;
        s.Hkv = a.Hkv;
        s.tu = 2 * p.tq;
        s.tile = p.tq;
        s.kb = kBN;
        s.start = kUnitStart;
        s.min_share = 2;  // a key tile for each side
        s.n_ctas = a.n_ctas;
        s.cap = a.max_history;
        ctas = a.n_ctas;
    } else {
        // Two row tiles share their K/V tiles; one alone makes twice as many units,
        // half as long.  The longest unit bounds a call with few, the work one with
        // many: which form ends first is reckoned from the rows (us: a key tile of
        // one or two row tiles, a unit's start and end, a third of a unit for CTAs
        // that end apart; causal units see half of the longest one's tiles on
        // average).  Measured, one against two, 16/2 heads of 128: 2500 rows 31.7,
        // 38.5; 4000 rows 61.9, 57.1; 8/8 heads of 64: 4000 rows 32.8, 56.8.
        const float tiles = float((int64_t(a.r.max_rows) + kBN - 1) / kBN);
        auto ends = [&](int tu, float tile) {
            const float units = float(a.Hkv) * float((int64_t(a.r.total_rows) + tu - 1) / tu);
            const float mean = tile * (tiles + 1.f) * 0.5f + 4.f;
            return std::max(tile * tiles + 4.f, units * mean / float(a.n_ctas) + mean / 3.f);
        };
        p.prompt = prompt_shape(a, ends(p.tq, 0.9f) < ends(2 * p.tq, 1.75f) ? p.tq : 2 * p.tq, kBN);
        ctas = prompt_numbers(p.prompt);
    }
    e = launch_pdl(kern, dim3(unsigned(ctas)), dim3(kThreads), Smem<D>::kBytes, st, mq, mk, mv, mkc, mvc, p);
    if (e != cudaSuccess || !kTree) return e;
    return launch_join<TOut, D>(p.shape, a, 2 * kBM, st);
}

template <typename T, int D> cudaError_t launch_out(const PackedAttn& a, cudaStream_t st) {
    if (a.out_dtype == PA_F32)
        return a.tree_mask ? launch_typed<T, D, true, float>(a, st) : launch_typed<T, D, false, float>(a, st);
    return a.tree_mask ? launch_typed<T, D, true, T>(a, st) : launch_typed<T, D, false, T>(a, st);
}

}  // namespace

size_t tree_tc_workspace_bytes(int D, int n_ctas) { return tree_workspace_bytes(2 * kBM, D, n_ctas); }

cudaError_t launch_packed_tc(const PackedAttn& a, cudaStream_t st) {
    if (a.dtype == PA_BF16)
        return a.D == 64 ? launch_out<__nv_bfloat16, 64>(a, st) : launch_out<__nv_bfloat16, 128>(a, st);
    return a.D == 64 ? launch_out<__half, 64>(a, st) : launch_out<__half, 128>(a, st);
}

}  // namespace pa
