// pa_key_weights_tc.cu -- key weights of many columns (rows x heads) of a
// 16-bit type, on the tensor cores.
//
// Both passes multiply a tile A of 128 rows, which stays, with tiles B of 128
// rows that stream past it, and reduce along B.  A is on the accumulator's 128
// lanes, so a thread reduces its own lane's columns and nothing crosses lanes:
//   statistics: A = 128 columns (128 / G rows of q, all G heads of the kv
//               head), B = the keys; a running maximum and sum a lane
//   gathering:  A = 128 keys, B = the columns; sum of 2^(s - m - log2 l) a lane
// So Q K^T is computed twice, and no score leaves the SM.
//
// Two CTAs an SM, each with two groups of four warps for the scores, which take
// the B tiles in turn, one warp that loads (TMA) and one that multiplies (two
// accumulators of 128 columns of tensor memory, one a group): while one CTA
// begins or ends a unit, the other computes, and four warps to a scheduler hide
// one another's latencies (one group: 58 and 69 us for the passes of four prompts
// of 2560 rows and less).  A score takes a multiply-add, an exponential and an
// addition in each pass, and 128 x 128 of them take longer than their product; yet no
// pipe is saturated (special functions 42% and 32% busy, an SM's throughput 52% and
// 42%): a warp waits for each chunk's load from tensor memory before it begins with
// the chunk, so that latency and the order of a warp's own steps bound it.  A column's m and l
// go into one number, m + log2 l, which all lanes read from shared memory: with
// two, 16 bytes for two scores, those reads bounded the second pass (92 us against
// the first's 59, four prompts of 2560 rows and less).  Its rounding, 2^-18 where m
// is below 128, goes into the column's weights.  Columns of larger scores, of which
// it would take more and at last all of log2 l, keep both numbers, and their chunk
// goes another way (which costs the others 2%: 114.0 -> 116.8 us).
//
// Units (an A tile with all its B tiles) are laid on a line, sequence by
// sequence and kv head by kv head, each as long as it costs, and the line is cut
// into equal shares, one a CTA.  Causal units get longer or shorter along the
// sequence; the i-th is followed by the i-th from the end, so that a pair's
// length is the same for all of them and a place on the line is found by
// division.  A unit inside one share is finished there; the pieces of others
// are joined in ascending order by a kernel of its own.
//
// Four prompts of 2560, 130, 1999 and 37 rows, 32/8 heads of 128, bf16: 117 us, 53
// for the statistics and 67 for the gathering when each runs by itself; 43.3 GFLOP of
// products twice over are 46 us at the measured rate of a large bf16 product.
#include <type_traits>

#include "pa_device.h"
#include "pa_key_weights.h"
#include "pa_pairs.cuh"
#include "pa_tc.cuh"
#include "pa_tmap.h"

namespace pa {

namespace {

constexpr int kTile = 128;
constexpr int kThr = 320;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kPerSm = 2;          // CTAs (one: 135 us for the four prompts instead of 114)
constexpr int kStart = 2;          // what beginning and ending a unit costs, in B tiles (4: 118 us, 1: the same)
constexpr int kMinShare = 4;       // of the line, a CTA (300 rows, 64/8 heads: 22 us; 1: 24, 12: 31)
constexpr uint32_t kHalf = kTile * 128;  // bytes of 64 dims of a tile
constexpr uint32_t kNegInf = 0xff800000u;
constexpr float kFar = 128.f;      // largest scores (base 2, scaled) below it: m + log2 l is off by 2^-18 at most
constexpr int kFarColumn = -2;     // among a chunk's limits: a column of larger ones
constexpr uint64_t kWaitNs = 2000000000ull;  // a role gives up after 2 s on one barrier
constexpr uint32_t kSleepNs = 20000;

template <int D> struct Smem {
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr uint32_t kTileBytes = kTile * D * 2;
    static constexpr uint32_t kB = kTileBytes;
    static constexpr uint32_t kStats = kB + kStages * kTileBytes;  // [group][3][128] of -(m + log2 l), or -m
    static constexpr uint32_t kFactors = kStats + 6 * 128 * 4;     // [2][3][128] 1, or 1 / l
    static constexpr uint32_t kLimits = kFactors + 6 * 128 * 4;    // [2][3][128] last key that a column sees
    static constexpr uint32_t kChunks = kLimits + 6 * 128 * 4;     // [2][3][4][2] lowest and highest of 32 columns'
    static constexpr uint32_t kHelp = kChunks + 6 * 4 * 2 * 4;     // [2][128] what a group leaves for the other
    static constexpr uint32_t kBars = kHelp + 2 * 128 * 8;
    static constexpr int kNumBars = 2 + 2 * kStages + 4 + 6 + 4 + 2;
    static constexpr uint32_t kBytes = 1024 + kBars + kNumBars * 8 + 16;
};

struct WideArgs {
    KwArgs a;
    int32_t tq, workers, head_first;
    float* logs;          // [2][total_rows][Hq] of log_of
    int64_t columns;      // total_rows Hq
    float2* parts_stats;  // [2 workers][128]
    float* parts_sums;    // [2 workers][128]
};

// ---- the line of units ------------------------------------------------------------
struct Line {
    int T, L, before, row0;
    int flat, tri;      // units of equal length, then units in pairs
    int flat_cost;
    int pair, len;      // positions of a pair, of a kv head (below 2^30: the host sees to that)
};

// Length of unit u.
template <int kPass> __device__ inline int tiles_of(const WideArgs& w, const Line& q, int u) {
    if (kPass == 0) return (q.before + min(q.T, (u + 1) * w.tq) + kTile - 1) / kTile;
    return (q.T + w.tq - 1) / w.tq - max(0, kTile * u - q.before) / w.tq;
}
// The first B tile of unit u.
template <int kPass> __device__ inline int first_of(const WideArgs& w, const Line& q, int u) {
    return kPass == 0 ? 0 : max(0, kTile * u - q.before) / w.tq;
}

template <int kPass> __device__ inline Line line_of(const WideArgs& w, int s) {
    Line q = {};
    if (s >= w.a.num_seqs) return q;
    const KwSeq k = kw_seq(w.a, s);
    q.T = k.T;
    q.L = k.L;
    q.row0 = k.row0;
    q.before = k.L - k.T;
    if (k.T == 0) return q;
    const int nq = (k.T + w.tq - 1) / w.tq, nk = (k.L + kTile - 1) / kTile;
    // (sums of twice 2^30 and a few tiles fit in 32 bits without a sign)
    if (kPass == 0) {
        q.tri = nq;
        // the sum of two floors is at most the floor of the sum
        q.pair = 2 * kStart + int((2u * unsigned(q.before) + unsigned(nq + 1) * w.tq + 2u * (kTile - 1)) / kTile);
    } else {
        q.flat = min(nk, (q.before + w.tq - 1) / kTile + 1);
        q.flat_cost = kStart + nq;
        q.tri = nk - q.flat;
        if (q.tri)
            q.pair = 2 * kStart + 2 * nq + 1 -
                     int((unsigned(kTile) * (2u * q.flat + q.tri - 1u) - 2u * unsigned(q.before)) / w.tq);
    }
    q.len = q.flat * q.flat_cost + (q.tri + 1) / 2 * q.pair;
    return q;
}
// A unit, or its part in a share: B tiles [b0, b1).  Walks along the line: the
// units of a kv head, head by head, sequence by sequence.
struct Part {
    Line q;
    int s, g, unit;
    int64_t begin, end;  // the unit on the line
    int b0, b1;
    bool begins, whole;
    // the place of the unit: its number among those of equal length, or its pair and which of it
    int pair, second;
    int64_t pair_end;
};

template <int kPass> __device__ inline void set_unit(const WideArgs& w, Part& p) {
    if (p.pair < 0) {
        p.end = p.begin + p.q.flat_cost;
        return;
    }
    const int far = p.q.tri - 1 - p.pair;  // the longer one first
    p.unit = p.q.flat + ((kPass == 0) == (p.second == 0) ? far : p.pair);
    p.end = p.begin + kStart + tiles_of<kPass>(w, p.q, p.unit);
}
// The first unit of the kv head that begins at p.begin.
template <int kPass> __device__ inline void first_unit(const WideArgs& w, Part& p) {
    p.unit = 0;
    p.pair = p.q.flat ? -1 : 0;
    p.second = 0;
    p.pair_end = p.begin + p.q.pair;
    set_unit<kPass>(w, p);
}
// The unit behind p's; the line's end lies behind every share, so there is one
// wherever a share goes on.
template <int kPass> __device__ inline void next_unit(const WideArgs& w, Part& p) {
    if (p.pair < 0 && p.unit + 1 < p.q.flat) {
        p.begin = p.end;
        ++p.unit;
    } else if (p.pair >= 0 && !p.second && p.pair != p.q.tri - 1 - p.pair) {
        p.begin = p.end;
        p.second = 1;
    } else if (p.pair + 1 < (p.q.tri + 1) / 2) {  // the first or the next pair
        p.begin = p.pair < 0 ? p.end : p.pair_end;
        ++p.pair;
        p.second = 0;
        p.pair_end = p.begin + p.q.pair;
    } else {
        p.begin = p.pair < 0 ? p.end : p.pair_end;
        if (++p.g == w.a.Hkv) {
            p.g = 0;
            do p.q = line_of<kPass>(w, ++p.s);
            while (p.q.len == 0 && p.s < w.a.num_seqs);
        }
        first_unit<kPass>(w, p);
        return;
    }
    set_unit<kPass>(w, p);
}

// The share of worker i of a line (whole warp): its first place and, behind it,
// its last; the unit at its first place.  False where the share is empty.
template <int kPass>
__device__ inline bool share_of(const WideArgs& w, int i, int lane, int64_t& share, int64_t& x0, int64_t& x1,
                                int64_t& total, Part& p, bool at_end = false) {
    // lengths of 32 sequences at a time, kept for the search where there are no more
    int64_t v = 0, n = 0;
    total = 0;
    auto scan = [&](int s0) {
        n = int64_t(line_of<kPass>(w, s0 + lane).len) * w.a.Hkv;
        v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
    };
    for (int s0 = 0; s0 < w.a.num_seqs; s0 += 32) {
        scan(s0);
        total += __shfl_sync(0xffffffffu, v, 31);
    }
    const int64_t even = total + w.workers - 1;
    share = (even >> 31) == 0 ? int64_t(unsigned(even) / unsigned(w.workers)) : even / w.workers;
    if (share < kMinShare) share = kMinShare;
    x0 = share * i;
    x1 = min(total, x0 + share);
    if (x0 >= x1) return false;
    const int64_t x = at_end ? x1 - 1 : x0;
    int64_t in = x;
    p.s = 0;
    for (int s0 = 0; s0 < w.a.num_seqs; s0 += 32) {
        if (w.a.num_seqs > 32) scan(s0);
        const unsigned m = __ballot_sync(0xffffffffu, in < v);
        if (m) {
            const int l = __ffs(m) - 1;
            p.s = s0 + l;
            in -= __shfl_sync(0xffffffffu, v - n, l);
            break;
        }
        in -= __shfl_sync(0xffffffffu, v, 31);
    }
    p.q = line_of<kPass>(w, p.s);
    p.g = (in >> 31) == 0 ? int(unsigned(in) / unsigned(p.q.len)) : int(in / p.q.len);
    int off = int(in - int64_t(p.g) * p.q.len);
    const int flat_len = p.q.flat * p.q.flat_cost;
    p.unit = 0;
    p.second = 0;
    if (off < flat_len) {
        p.pair = -1;
        p.unit = off / p.q.flat_cost;
        p.begin = x - (off - p.unit * p.q.flat_cost);
        p.pair_end = 0;
        set_unit<kPass>(w, p);
    } else {
        off -= flat_len;
        p.pair = off / p.q.pair;
        p.begin = x - (off - p.pair * p.q.pair);
        p.pair_end = p.begin + p.q.pair;
        set_unit<kPass>(w, p);
        if (x >= p.end && p.pair != p.q.tri - 1 - p.pair) {
            p.begin = p.end;
            p.second = 1;
            set_unit<kPass>(w, p);
        }
    }
    return true;
}
// The part of the share's end [x, x1) that lies in p's unit, or in the next one
// where x is behind it; x moves behind the part.  False where there is no tile in it.
template <int kPass>
__device__ inline bool next_part(const WideArgs& w, int64_t& x, int64_t x1, Part& p) {
    if (x >= p.end) {
        next_unit<kPass>(w, p);
        if (x < p.begin) x = p.begin;
        if (x >= x1) return false;
    }
    const int64_t stop = min(p.end, x1);
    const int off = int(x - p.begin);
    p.begins = off == 0;
    p.whole = p.begins && stop == p.end;
    const int first = first_of<kPass>(w, p.q, p.unit);
    p.b0 = first + max(0, off - kStart);
    p.b1 = first + max(0, int(stop - p.begin) - kStart);
    x = stop;
    return p.b1 > p.b0;
}

// ---- waits ------------------------------------------------------------------------
__device__ inline bool wait_bar(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, kSleepNs)) return true;
        if (*abort_flag || globaltimer_ns() - t0 > kWaitNs) return false;
    }
}
__device__ inline bool wait_warp(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
}
__device__ inline void raise_abort(volatile uint32_t* abort_flag, uint32_t* dev_status) {
    *abort_flag = 1u;
    flag(dev_status, PA_DEV_TIMEOUT);
}

__device__ inline float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ inline uint64_t pair_of(uint32_t lo, uint32_t hi) {
    return pairs::pack(__uint_as_float(lo), __uint_as_float(hi));
}

// A column's weights are 2^(s - x) y: (m + log2 l, 1), or, where that sum would lose
// what matters of log2 l, (m, 1 / l).  x = -infinity: the column saw nothing.
__device__ inline float2 log_of(float m, float l) {
    if (l == 0.f) return make_float2(-INFINITY, 1.f);
    return fabsf(m) < kFar ? make_float2(m + log2f(l), 1.f) : make_float2(m, 1.f / l);
}
__device__ inline void set_log(const WideArgs& w, int64_t column, float m, float l) {
    const float2 x = log_of(m, l);
    w.logs[column] = x.x;
    w.logs[w.columns + column] = x.y;
}

// 32 scores of a lane: the running maximum (base 2, scaled), whether it is far, and the
// sum.  `real`: the lane's result is used.  A far maximum is a rounded product, and so are the scores that it is
// taken from: a product that is not rounded can lie half a step of m beside it, which at
// 2^30 is more than an exponent has room for.
__device__ inline void take(float& m, bool& far, uint64_t& l, uint64_t& l2, const uint32_t (&r)[32], float scale,
                            bool real) {
    float top = __uint_as_float(r[0]);
#pragma unroll
    for (int i = 1; i < 31; i += 2) top = max3(top, __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
    top = fmaxf(top, __uint_as_float(r[31])) * scale;
    if (top > m) {
        const float down = ex2(m - top);
        const uint64_t down2 = pairs::pack(down, down);
        l = pairs::mul(l, down2);
        l2 = pairs::mul(l2, down2);
        m = top;
        far = real && fabsf(m) >= kFar;
    }
    if (far) {
        // one by one: a paired product and sum become one operation, rounded once
        auto term = [&](uint32_t v) { return ex2(__fsub_rn(__fmul_rn(__uint_as_float(v), scale), m)); };
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            l = pairs::add(l, pairs::pack(term(r[i]), term(r[i + 1])));
            l2 = pairs::add(l2, pairs::pack(term(r[i + 2]), term(r[i + 3])));
        }
        return;
    }
    const uint64_t k = pairs::pack(scale, scale), minus = pairs::pack(-m, -m);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float2 x = pairs::unpack(pairs::fma(pair_of(r[i], r[i + 1]), k, minus));
        const float2 y = pairs::unpack(pairs::fma(pair_of(r[i + 2], r[i + 3]), k, minus));
        l = pairs::add(l, pairs::pack(ex2(x.x), ex2(x.y)));
        l2 = pairs::add(l2, pairs::pack(ex2(y.x), ex2(y.y)));
    }
}

// A score's weight where its column or a neighbour has a far maximum.  Above 1 only
// where the two passes' products would differ; a NaN stays one.
__device__ inline float far_weight(uint32_t v, float scale, float x, float y) {
    const float e = ex2(__fadd_rn(__fmul_rn(__uint_as_float(v), scale), x));
    return (e > 1.f ? 1.f : e) * y;
}

template <int kPass, typename T, int D>
__global__ void __launch_bounds__(kThr, kPerSm)
    wide_pass(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ WideArgs w) {
    using S = Smem<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int kStages = S::kStages, kHalves = D / 64;
    const KwArgs& a = w.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + S::kBars);
    uint64_t* a_full = bars;
    uint64_t* a_empty = bars + 1;
    uint64_t* b_full = bars + 2;
    uint64_t* b_empty = b_full + kStages;
    uint64_t* s_full = b_empty + kStages;
    uint64_t* s_empty = s_full + 2;
    uint64_t* st_full = s_empty + 2;  // [group][3], gathering: the columns' statistics written
    uint64_t* help_full = st_full + 6;
    uint64_t* help_empty = help_full + 2;
    uint64_t* mma_done = help_empty + 2;  // every product of the CTA has finished
    uint64_t* never = mma_done + 1;       // never arrived on: the debug_timeout wait
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + S::kNumBars);
    volatile uint32_t* abort_flag = tslot + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(a_full, 1);
        mbar_init(a_empty, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&b_full[i], 1);
            mbar_init(&b_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 4);
            for (int j = 0; j < 3; ++j) mbar_init(&st_full[3 * i + j], 4);
            mbar_init(&help_full[i], 4);
            mbar_init(&help_empty[i], 4);
        }
        mbar_init(mma_done, 1);
        mbar_init(never, 1);
        *abort_flag = 0u;
        mbar_fence_init();
    }
    if (kPass == 0) {
        pdl_wait_primary();
        pdl_launch_dependents();
        if (blockIdx.x == 0)
            for (int s = tid; s < a.num_seqs; s += kThr)
                if (kw_seq(a, s).bad) flag(a.dev_status, PA_DEV_BAD_LEN);
    }
    int64_t share, x0, x1, total;
    Part p;
    const bool any = share_of<kPass>(w, blockIdx.x, lane, share, x0, x1, total, p);
    if (kPass == 1) {  // the lengths were there before the first kernel let others start
        pdl_wait_primary();
        pdl_launch_dependents();
    }
    if (!any) return;  // the whole CTA, before any barrier
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tslot, 256);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *tslot;
    if (a.debug_timeout) {
        // Testing: a wait that runs out before any copy is issued aborts every role.
        if (tid == 0 && !mbar_wait_ns(never, 0, 0)) raise_abort(abort_flag, a.dev_status);
        __syncthreads();
    }
    bool ok = !*abort_flag;
    const int P = a.page_size, PT = kTile / P;

    if (warp == kLoadWarp) {
        const uint32_t q_bytes = uint32_t(kHalves) * 128u * uint32_t(a.G * w.tq);
        auto load_q = [&](uint8_t* dst, uint64_t* bar, const Part& p, int i) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, q_bytes);
                for (int h = 0; h < kHalves; ++h)
                    tma_load_3d(dst + h * kHalf, &tmQ, bar, 64 * h, p.g * a.G, p.q.row0 + i * w.tq);
            }
            __syncwarp();
        };
        auto load_k = [&](uint8_t* dst, uint64_t* bar, const Part& p, int j) {
            // lane l: page l of the tile; none: beyond the tensor, so that the box reads as zeros
            int pg = a.num_pages;
            const int at = j * PT + lane;
            if (lane < PT && at * P < p.q.L) {
                const int e = a.block_tables[int64_t(p.s) * a.max_blocks + at];
                if (e >= 0 && e < a.num_pages)
                    pg = e;
                else if (kPass == 0)
                    flag(a.dev_status, PA_DEV_BAD_PAGE);
            }
            if (lane == 0) mbar_arrive_expect_tx(bar, S::kTileBytes);
            __syncwarp();
            if (lane < PT)
                for (int h = 0; h < kHalves; ++h)
                    tma_load_4d(dst + h * kHalf + lane * P * 128, &tmK, bar, 64 * h, w.head_first ? p.g : 0,
                                w.head_first ? 0 : p.g, pg);
        };
        int n = 0, parts = 0;
        for (int64_t x = x0; ok && x < x1;) {
            if (!next_part<kPass>(w, x, x1, p)) continue;
            if (parts) ok = wait_warp(a_empty, (parts - 1) & 1, abort_flag);
            if (!ok) break;
            if (kPass == 0)
                load_q(base, a_full, p, p.unit);
            else
                load_k(base, a_full, p, p.unit);
            ++parts;
            for (int b = p.b0; b < p.b1; ++b, ++n) {
                const int st = n % kStages;
                if (n >= kStages) ok = wait_warp(&b_empty[st], ((n / kStages) - 1) & 1, abort_flag);
                if (!ok) break;
                uint8_t* dst = base + S::kB + st * S::kTileBytes;
                if (kPass == 0)
                    load_k(dst, &b_full[st], p, b);
                else
                    load_q(dst, &b_full[st], p, b);
            }
        }
        if (lane == 0) {
            if (!ok) raise_abort(abort_flag, a.dev_status);
            // never leave the CTA with copies in flight
            for (int i = max(0, n - kStages); i < n; ++i) mbar_wait_ns(&b_full[i % kStages], (i / kStages) & 1, kWaitNs);
            if (parts) mbar_wait_ns(a_full, (parts - 1) & 1, kWaitNs);
        }
    } else if (warp == kMmaWarp) {
        const uint32_t idesc = tc::idesc_f16(kTile, kTile, kBf16, false), hi = tc::desc_hi_sw128(1024);
        const uint32_t a_lo = tc::desc_lo(smem_u32(base), 16), b_lo = tc::desc_lo(smem_u32(base + S::kB), 16);
        int n = 0, parts = 0;
        for (int64_t x = x0; ok && x < x1;) {
            if (!next_part<kPass>(w, x, x1, p)) continue;
            ok = wait_warp(a_full, parts & 1, abort_flag);
            ++parts;
            for (int b = p.b0; ok && b < p.b1; ++b, ++n) {
                const int st = n % kStages, buf = n & 1;
                ok = wait_warp(&b_full[st], (n / kStages) & 1, abort_flag);
                if (ok && n >= 2) ok = wait_warp(&s_empty[buf], ((n >> 1) - 1) & 1, abort_flag);
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t bx = b_lo + st * (S::kTileBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                    tc::mma_ss_elect(tm + 128 * buf, tc::make_desc(a_lo + off, hi), tc::make_desc(bx + off, hi), idesc,
                                     ks > 0);
                }
                tc::commit_elect(&b_empty[st]);
                if (b + 1 == p.b1) tc::commit_elect(a_empty);
                tc::commit_elect(&s_full[buf]);
            }
        }
        if (!ok && lane == 0) raise_abort(abort_flag, a.dev_status);
        // tensor memory is not freed, nor the operands' shared memory left, under a product
        tc::commit_elect(mma_done);
        if (!__all_sync(0xffffffffu, mbar_wait_ns(mma_done, 0, kWaitNs)) && lane == 0)
            flag(a.dev_status, PA_DEV_TIMEOUT);
    } else {
        const int group = warp >> 2, row = tid & 127;  // the group's accumulator and buffers, the thread's lane of A
        float* sm_stats = reinterpret_cast<float*>(base + S::kStats) + 384 * group;
        float* sm_factors = reinterpret_cast<float*>(base + S::kFactors) + 384 * group;
        int* sm_limits = reinterpret_cast<int*>(base + S::kLimits) + 384 * group;
        int* sm_chunks = reinterpret_cast<int*>(base + S::kChunks) + 24 * group;
        float2* sm_help = reinterpret_cast<float2*>(base + S::kHelp);
        const uint32_t acc_at = tm + 128 * group + (uint32_t(warp & 3) << 21);
        const int cols = w.tq * a.G;
        const int my_t = row / a.G, my_h = row - my_t * a.G;
        int n = 0, seen = 0;           // tiles of the CTA before the part, of the group so far
        int buf = 0, turn = 0;         // seen % 3 and the parity of seen / 3
        int helped = 0, was_helped = 0;  // parts that the group left to the other, and the other to it
        for (int64_t x = x0; ok && x < x1;) {
            if (!next_part<kPass>(w, x, x1, p)) continue;
            const int tiles = p.b1 - p.b0, first = (group + n) & 1;  // the group's first tile of the part
            const bool ends = first == 0;  // it has the part's first tile and writes its result
            n += tiles;
            if (first >= tiles) continue;
            float m = kLowestScore, sum = 0.f;
            bool far = false;
            uint64_t acc = 0, acc2 = 0;  // two sums each
            const int32_t* table = a.block_tables + int64_t(p.s) * a.max_blocks;
            // statistics: the lane's column; gathering: the lane's key
            const int t = p.unit * w.tq + my_t;
            const int key = kTile * p.unit + row;
            auto stat_at = [&](int tt) { return w.logs + (int64_t(p.q.row0 + tt) * a.Hq + p.g * a.G + my_h); };
            auto column = [&](int b) {  // the first number of log_of the thread's column of Q tile b
                const int tt = b * w.tq + my_t;
                return row < cols && tt < p.q.T ? *stat_at(tt) : -INFINITY;
            };
            auto pages = [&](int b) {  // a lane of PT: the tile's page
                const int at = b * PT + lane;
                return lane < PT && at * P < p.q.L ? table[at] : -1;
            };
            // The statistics of a tile's columns, to be read by the whole group: written
            // a tile ahead, in three buffers.  Whoever writes tile i + 1's has waited for
            // all warps to write tile i's, which each does after it has waited for tile
            // i - 1's, or once a part's last tile is done: so all are through with
            // tile i - 2, whose buffer it is.
            auto show = [&](int b, float log, int to) {
                const int lim = log == -INFINITY ? -1 : p.q.before + b * w.tq + my_t;  // a NaN counts as seen
                const bool far = lim >= 0 && fabsf(log) >= kFar;
                sm_stats[128 * to + row] = -log;
                sm_factors[128 * to + row] = far ? stat_at(b * w.tq + my_t)[w.columns] : 1.f;
                sm_limits[128 * to + row] = lim;
                const int low = __reduce_min_sync(0xffffffffu, far ? kFarColumn : lim);
                const int high = __reduce_max_sync(0xffffffffu, lim);
                if (lane == 0) {
                    sm_chunks[8 * to + 2 * (warp & 3)] = low;
                    sm_chunks[8 * to + 2 * (warp & 3) + 1] = high;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&st_full[3 * group + to]);
            };
            float ahead = -INFINITY;
            int page_ahead = -1;
            if (kPass == 1) {
                const float log = column(p.b0 + first);
                if (p.b0 + first + 2 < p.b1) ahead = column(p.b0 + first + 2);
                show(p.b0 + first, log, buf);
            } else {
                page_ahead = pages(p.b0 + first);
            }
            for (int b = p.b0 + first; b < p.b1; b += 2, ++seen) {
                uint32_t page_bits = 0;
                if (kPass == 1) {
                    ok = wait_warp(&st_full[3 * group + buf], turn, abort_flag);
                    if (!ok) break;
                    if (b + 2 < p.b1) {
                        show(b + 2, ahead, buf == 2 ? 0 : buf + 1);
                        if (b + 4 < p.b1) ahead = column(b + 4);
                    }
                } else {
                    page_bits = __ballot_sync(0xffffffffu, page_ahead >= 0 && page_ahead < a.num_pages);
                    if (b + 2 < p.b1) page_ahead = pages(b + 2);
                }
                ok = wait_warp(&s_full[group], seen & 1, abort_flag);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tc::ld_32x32b_x32(acc_at + 32 * c, v);
                    tc::wait_ld();
                    tc::reg_fence(v);
                    if (c == 3) {
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_empty[group]);
                    }
                    if (kPass == 0) {
                        // keys 32 c .. 32 c + 31 of the tile: seen by all lanes, or a bit for each
                        const int k0 = kTile * b + 32 * c;
                        const uint32_t mine = P == 32 ? (page_bits >> c) & 1u : (page_bits >> (2 * c)) & 3u;
                        const bool all = mine == (P == 32 ? 1u : 3u) && k0 + 31 <= p.q.before + p.unit * w.tq;
                        if (!all) {
                            const int upto = p.q.before + t - k0 + 1;
                            uint32_t bits = upto >= 32 ? 0xffffffffu : upto <= 0 ? 0u : (1u << upto) - 1u;
                            bits &= P == 32 ? (mine ? 0xffffffffu : 0u)
                                            : ((mine & 1u) ? 0xffffu : 0u) | ((mine & 2u) ? 0xffff0000u : 0u);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = (bits >> i) & 1u ? v[i] : kNegInf;
                        }
                        take(m, far, acc, acc2, v, a.scale_log2, row < cols);
                    } else {
                        const int low = sm_chunks[8 * buf + 2 * c], high = sm_chunks[8 * buf + 2 * c + 1];
                        if (high < kTile * p.unit) continue;  // no column sees a key of the tile
                        const float4* st = reinterpret_cast<const float4*>(sm_stats + 128 * buf + 32 * c);
                        const uint64_t k = pairs::pack(a.scale_log2, a.scale_log2);
                        if (low >= kTile * p.unit + kTile - 1) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 y = st[i / 4];
                                const float2 e = pairs::unpack(pairs::fma(pair_of(v[i], v[i + 1]), k, pairs::pack(y.x, y.y)));
                                const float2 f = pairs::unpack(pairs::fma(pair_of(v[i + 2], v[i + 3]), k, pairs::pack(y.z, y.w)));
                                acc = pairs::add(acc, pairs::pack(ex2(e.x), ex2(e.y)));
                                acc2 = pairs::add(acc2, pairs::pack(ex2(f.x), ex2(f.y)));
                            }
                        } else if (low != kFarColumn) {
                            const int* lim = sm_limits + 128 * buf + 32 * c;
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 y = st[i / 4];
                                const int4 last4 = *reinterpret_cast<const int4*>(lim + i);
                                const float e0 = ex2(fmaf(__uint_as_float(v[i]), a.scale_log2, y.x));
                                const float e1 = ex2(fmaf(__uint_as_float(v[i + 1]), a.scale_log2, y.y));
                                const float e2 = ex2(fmaf(__uint_as_float(v[i + 2]), a.scale_log2, y.z));
                                const float e3 = ex2(fmaf(__uint_as_float(v[i + 3]), a.scale_log2, y.w));
                                sum += (key <= last4.x ? e0 : 0.f) + (key <= last4.y ? e1 : 0.f);
                                sum += (key <= last4.z ? e2 : 0.f) + (key <= last4.w ? e3 : 0.f);
                            }
                        } else {
                            const float4* factors = reinterpret_cast<const float4*>(sm_factors + 128 * buf + 32 * c);
                            const int* lim = sm_limits + 128 * buf + 32 * c;
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 y = st[i / 4], f = factors[i / 4];
                                const int4 last4 = *reinterpret_cast<const int4*>(lim + i);
                                if (key <= last4.x) sum += far_weight(v[i], a.scale_log2, y.x, f.x);
                                if (key <= last4.y) sum += far_weight(v[i + 1], a.scale_log2, y.y, f.y);
                                if (key <= last4.z) sum += far_weight(v[i + 2], a.scale_log2, y.z, f.z);
                                if (key <= last4.w) sum += far_weight(v[i + 3], a.scale_log2, y.w, f.w);
                            }
                        }
                    }
                }
                if (++buf == 3) {
                    buf = 0;
                    turn ^= 1;
                }
            }
            if (!ok) break;
            const float2 two = pairs::unpack(pairs::add(acc, acc2));
            sum += two.x + two.y;
            if (!ends) {  // leave it to the group that has the first tile
                if (helped) ok = wait_warp(&help_empty[group], (helped - 1) & 1, abort_flag);
                if (!ok) break;
                ++helped;
                sm_help[128 * group + row] = make_float2(m, sum);
                __syncwarp();
                if (lane == 0) mbar_arrive(&help_full[group]);
                continue;
            }
            if (tiles > 1) {
                ok = wait_warp(&help_full[group ^ 1], was_helped & 1, abort_flag);
                if (!ok) break;
                ++was_helped;
                const float2 other = sm_help[128 * (group ^ 1) + row];
                __syncwarp();
                if (lane == 0) mbar_arrive(&help_empty[group ^ 1]);
                if (kPass == 0)
                    kw_join(m, sum, other.x, other.y);
                else
                    sum += other.y;
            }
            if (kPass == 0) {
                if (!p.whole)
                    w.parts_stats[(2 * int64_t(blockIdx.x) + p.begins) * kTile + row] = make_float2(m, sum);
                else if (row < cols && t < p.q.T)
                    set_log(w, int64_t(p.q.row0 + t) * a.Hq + p.g * a.G + my_h, m, sum);
            } else {
                bool there = false;
                if (key < p.q.L) {
                    const int pg = table[key >> a.page_shift];
                    there = pg >= 0 && pg < a.num_pages;
                }
                if (!there) sum = 0.f;
                if (!p.whole) {
                    w.parts_sums[(2 * int64_t(blockIdx.x) + p.begins) * kTile + row] = sum;
                } else if (key < p.q.L) {
                    float* to = a.weights + (int64_t(p.s) * a.Hkv + p.g) * a.slots + key;
                    if (a.decay > 0.f && key < p.q.before) sum += a.decay * *to;
                    *to = sum;
                }
            }
        }
        if (!ok && lane == 0) raise_abort(abort_flag, a.dev_status);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tm, 256);
    }
}

// A CTA for each share: the unit that begins in it and ends behind it.
template <int kPass> __global__ void __launch_bounds__(kTile) wide_join(const __grid_constant__ WideArgs w) {
    const KwArgs& a = w.a;
    const int tid = threadIdx.x, lane = tid & 31;
    int64_t share, x0, x1, total;
    Part p;
    // the unit at the share's last place; the lengths were there before the first kernel let others start
    if (kPass == 0) pdl_launch_dependents();  // the second pass reads nothing else before this kernel's end
    const bool any = share_of<kPass>(w, blockIdx.x, lane, share, x0, x1, total, p, true);
    pdl_wait_primary();
    if (kPass == 1) pdl_launch_dependents();
    if (!any || x1 >= total || p.end <= x1 || p.begin < x0) return;  // none, whole, or another CTA's
    float m = kLowestScore, l = 0.f;
    for (int i = blockIdx.x; i < w.workers && i * share < p.end; ++i) {
        if (min(p.end, (i + 1) * share) <= p.begin + kStart) continue;  // no tile in this share
        const int slot = (2 * i + (i == int(blockIdx.x))) * kTile + tid;
        if (kPass == 0)
            kw_join(m, l, w.parts_stats[slot].x, w.parts_stats[slot].y);
        else
            l += w.parts_sums[slot];
    }
    if (kPass == 0) {
        const int t = p.unit * w.tq + tid / a.G;
        if (tid < w.tq * a.G && t < p.q.T)
            set_log(w, int64_t(p.q.row0 + t) * a.Hq + p.g * a.G + tid % a.G, m, l);
    } else {
        const int key = kTile * p.unit + tid;
        if (key < p.q.L) {
            float* to = a.weights + (int64_t(p.s) * a.Hkv + p.g) * a.slots + key;
            if (a.decay > 0.f && key < p.q.before) l += a.decay * *to;
            *to = l;
        }
    }
}

template <typename T, int D>
cudaError_t launch_wide(const CUtensorMap& mq, const CUtensorMap& mk, const WideArgs& w, cudaStream_t st) {
    static std::atomic<uint64_t> done0{0}, done1{0};
    constexpr size_t smem = Smem<D>::kBytes;
    cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(wide_pass<0, T, D>), smem, done0);
    if (e == cudaSuccess) e = allow_shared_memory(reinterpret_cast<const void*>(wide_pass<1, T, D>), smem, done1);
    if (e == cudaSuccess) e = launch_pdl(wide_pass<0, T, D>, dim3(w.workers), dim3(kThr), smem, st, mq, mk, w);
    if (e == cudaSuccess) e = launch_pdl(wide_join<0>, dim3(w.workers), dim3(kTile), 0, st, w);
    if (e == cudaSuccess) e = launch_pdl(wide_pass<1, T, D>, dim3(w.workers), dim3(kThr), smem, st, mq, mk, w);
    if (e == cudaSuccess) e = launch_pdl(wide_join<1>, dim3(w.workers), dim3(kTile), 0, st, w);
    return e;
}

}  // namespace

size_t key_weights_tc_parts(int n_ctas) {
    return size_t(2 * kPerSm) * n_ctas * kTile * (sizeof(float2) + sizeof(float));
}

cudaError_t launch_key_weights_tc(const KwArgs& a, pa_dtype dt, int D, int n_ctas, void* parts, cudaStream_t st) {
    WideArgs w = {};
    w.a = a;
    w.tq = kTile / a.G;
    w.workers = kPerSm * n_ctas;
    w.head_first = a.head_stride <= a.token_stride;
    w.logs = reinterpret_cast<float*>(a.stats);
    w.columns = int64_t(a.total_rows) * a.Hq;
    w.parts_stats = static_cast<float2*>(parts);
    w.parts_sums = reinterpret_cast<float*>(w.parts_stats + size_t(2) * w.workers * kTile);
    CUtensorMap mq, mk;
    if (!tmap_rows(&mq, dt, a.q, D, a.Hq, a.total_rows, a.q_stride, a.G, w.tq) ||
        !tmap_pages(&mk, dt, a.k, D, a.Hkv, a.page_size, a.num_pages, a.head_stride, a.token_stride, a.page_stride,
                    w.head_first))
        return cudaErrorInvalidValue;
    if (dt == PA_BF16)
        return D == 64 ? launch_wide<__nv_bfloat16, 64>(mq, mk, w, st) : launch_wide<__nv_bfloat16, 128>(mq, mk, w, st);
    return D == 64 ? launch_wide<__half, 64>(mq, mk, w, st) : launch_wide<__half, 128>(mq, mk, w, st);
}

}  // namespace pa
