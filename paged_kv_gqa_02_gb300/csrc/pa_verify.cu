// pa_verify.cu -- which drafted tokens the target's distribution accepts, and
// the token behind them.
//
// A cluster of CTAs walks one sequence's tree.  Only the rows that the walk
// visits are read: their logits' largest value and sum in one pass (the
// draft's row in the same one), then scalars alone decide about the children.
// After k rejections what is left of p is max(p - a q, 0) / M with
//   a_1 = 1, M_k = sum max(p - a_k q, 0), a_{k+1} = a_k + M_k,
// which is k times "subtract q, clamp, normalise" in one step, so a rejection
// costs one sum over the vocabulary whatever came before it; the last child's
// none, and certain drafts' (q a single token) none.  The next token is the
// largest p_i / e_i for exponential e_i: a comparison of single terms, while a
// search in running sums would meet a border every few 2^-24 in a vocabulary's
// tail.  M does not matter to it.  A p is off by 2^-22 of its value at most for each
// unit of its exponent (x - top) c, which is rounded, and by some more for the sums;
// p - a q by that share of p and of a q, which is more of what is left.  Where the
// draft's row is the target's, nothing is left, exactly: p - a q is one expression
// everywhere, and its factor of the draft's exponentials, a times the sums' ratio, is
// a where the sums are equal.
//
// The walk's time is a chain of passes, each bound by latency: the exponentials
// of a row and one exchange, some 5 us together (64 chains of five drafts, 50021
// fp16 tokens: 7 passes, 39 us; one chain of four, 32000 fp32 tokens: 11 us; 16 trees
// of up to 63, 131072 bf16 tokens: 35 to 43 us).  One CTA a sequence
// that read rows from L2 took 232, 24 and 145 us.  The bytes, 24 MB for the chains,
// would take 4 us.  A CTA has a run of the vocabulary, and its part of
// the rows waits in shared memory: the row at hand, for all of its passes, and the
// first child's, on its way (bulk copies) while the parent's is summed and decided;
// the random numbers from the start.  For an exchange every warp sends its result
// to the shared memory of every CTA of the cluster, counted by an mbarrier there.  A
// warp of its own, the leader, orders the copies, reads what it needs of the
// children meanwhile, joins the results and orders the next pass; leaders of a
// cluster join the same in the same order and so decide the same.  Only rank 0
// writes.  A second kernel joins the sequences' lists.
#include <cooperative_groups.h>

#include "pa_cp_async.cuh"
#include "pa_device.h"
#include "pa_pairs.cuh"
#include "pa_ptx.cuh"
#include "pa_rows.cuh"
#include "pa_serving.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kThr = 512;          // of the passes; the leader's warp comes behind them
constexpr int kWarps = kThr / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxDrafts = 1024;  // rows of a sequence
constexpr int kPackThr = 1024;
constexpr uint64_t kWaitNs = 2000000000ull;  // an exchange gives up after 2 s
constexpr uint64_t kTestNs = 2000000ull;     // or, testing, after 2 ms
constexpr uint64_t kDrainNs = 1000000ull;    // what has been sent arrives within microseconds

// The largest logit and the sum of 2^((x - largest) c); with a NaN or an
// infinite largest one the sum is not finite.
struct Stat {
    float top, sum;
};
// What a warp found in a pass, in two parts of 16 bytes.
struct __align__(16) Stats {
    Stat p, q;
};
struct __align__(16) Pick {
    float key;  // of the best candidate for the next token, or a sum
    int at;     // where the largest logit (greedy) or the best candidate is
    int pad[2];
};
// What the leader wants next: the walk to go on to a row, the sum of what is left
// of p, the best candidate for the next token, or nothing more.
enum { kGo, kMass, kPick, kStop };
struct Order {
    int what, went, phase;    // phase: of the copies to the row's slots
    int dropped;              // certain drafts rejected
    float p_top, q_top, less; // what is left: left_of(2^((x - p_top) c), 2^((y - q_top) c), less)
};
// A thread's running Stat, the sum in two parts.
struct Run {
    float top;
    uint64_t sum;
};

// Whether p lies on a 16-byte boundary.
template <typename T> __device__ inline bool wide_at(const T* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Shared memory for a CTA's part of two rows and their drafts', and of the
// random numbers where they fit beside them: units of eight elements, in order.
// Units beyond the room come to the slots of units that are done with.
constexpr size_t kRoom = 203648;  // with what is laid out by the compiler, all that a CTA may have
template <typename T> constexpr int kParts = 8 / Elt<T>::kVec;  // 16-byte parts of a unit

// A whole number of 16 bytes between 16-byte boundaries, counted by the mbarrier.
__device__ inline void copy_bulk(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(to)),
                 "l"(from), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ inline void prefetch_bulk(const void* from, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

// Eight elements to a unit's slot.  Copies that arrive later, but for 16-bit
// elements off the 16-byte boundaries.
template <typename T> __device__ inline void stage8(uint4* slot, const T* p) {
    if (wide_at(p)) {
#pragma unroll
        for (int i = 0; i < 8 / Elt<T>::kVec; ++i)
            cp_async16(smem_u32(slot + i), reinterpret_cast<const uint4*>(p) + i);
    } else if (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) cp_async4(smem_u32(slot) + 4 * i, p + i);
    } else {
        const unsigned short* e = reinterpret_cast<const unsigned short*>(p);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = uint32_t(__ldg(e + 2 * i)) | uint32_t(__ldg(e + 2 * i + 1)) << 16;
        *slot = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// Eight numbers off the 16-byte boundaries, out of the three units of four that
// hold them where those lie inside [first, end).
__device__ inline void read8(const float* p, const float* first, const float* end, float (&x)[8]) {
    const int off = int(reinterpret_cast<uintptr_t>(p) & 15) / 4;
    const float* q = p - off;
    if (q < first || q + 12 > end) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __ldg(p + i);
        return;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(q)), b = __ldg(reinterpret_cast<const float4*>(q) + 1);
    const float4 c = __ldg(reinterpret_cast<const float4*>(q) + 2);
    const float y[11] = {a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = off == 1 ? y[i] : off == 2 ? y[i + 1] : y[i + 2];
}
template <typename T> __device__ inline void take_slot(const uint4* slot, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8 / Elt<T>::kVec; ++i) vec_to_f32<T>(slot[i], x + i * Elt<T>::kVec);
}
// The largest of a slot's eight; NaNs are passed over.  16-bit types two at a time.
template <typename T> __device__ inline float max_slot(const uint4* slot);
template <> __device__ inline float max_slot<float>(const uint4* slot) {
    float x[8];
    take_slot<float>(slot, x);
    return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}
template <> __device__ inline float max_slot<__half>(const uint4* slot) {
    const uint4 v = *slot;
    const __half2* h = reinterpret_cast<const __half2*>(&v);
    const float2 m = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
    return fmaxf(m.x, m.y);
}
template <> __device__ inline float max_slot<__nv_bfloat16>(const uint4* slot) {
    const uint4 v = *slot;
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
    const float2 m = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
    return fmaxf(m.x, m.y);
}

// 16 bytes to the same place of another CTA's shared memory, counted by its mbarrier.
__device__ inline void send16(uint32_t to, uint32_t bar, const uint4& v) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
        "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
        : "memory");
}
__device__ inline uint32_t in_cta(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Without branches: a largest value of -infinity stands for 0, so that
// -infinity adds nothing and a NaN is not lost.
__device__ inline float raise(Run& s, float top, float c) {
    const float now = fmaxf(s.top, top), ref = now > -INFINITY ? now : 0.f;
    const float down = ex2((s.top - ref) * c);
    s.sum = pairs::mul(s.sum, pairs::pack(down, down));
    s.top = now;
    return ref;
}
__device__ inline void add8(Run& s, const float (&x)[8], float ref, float c) {
    const uint64_t minus = pairs::pack(-ref, -ref), c2 = pairs::pack(c, c);
    uint64_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 d = pairs::unpack(pairs::mul(pairs::add(pairs::pack(x[2 * i], x[2 * i + 1]), minus), c2));
        e[i] = pairs::pack(ex2(d.x), ex2(d.y));
    }
    s.sum = pairs::add(s.sum, pairs::add(pairs::add(e[0], e[1]), pairs::add(e[2], e[3])));
}
__device__ inline void take1(Run& s, float x, float c) {
    const float ref = raise(s, x, c);
    s.sum = pairs::add(s.sum, pairs::pack(ex2((x - ref) * c), 0.f));
}

// The largest of the warp's values, none of them a NaN.
__device__ inline float max_over_warp(float v) {
    const int b = __float_as_int(v);
    const int m = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));  // the order of floats
    return __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
}
// A Stat's sum for another largest value.  One that saw nothing, or -infinity
// alone, has what it has: 0, or a NaN.
__device__ inline float sum_at(const Stat& s, float top, float c) {
    return s.top > -INFINITY ? s.sum * ex2((s.top - top) * c) : s.sum;
}
__device__ inline Stat over_warp(const Stat& s, float c) {
    const float top = max_over_warp(s.top);
    return Stat{top, warp_sum(sum_at(s, top, c))};
}
__device__ inline Stat over_warp(const Run& s, float c) {
    const float2 two = pairs::unpack(s.sum);
    return over_warp(Stat{s.top, two.x + two.y}, c);
}
__device__ inline bool usable(const Stat& s) {
    return s.top > -INFINITY && s.top < INFINITY && s.sum < INFINITY;  // false for a NaN
}
// What rejections left of a target's exponential: a draft's takes `less` of it.
__device__ inline float left_of(float ex, float ey, float less) { return fmaxf(fmaf(-ey, less, ex), 0.f); }
__device__ inline void better(float& key, int& at, float key2, int at2) {
    if (key2 > key || (key2 == key && at2 < at)) {
        key = key2;
        at = at2;
    }
}
__device__ inline void better_over_warp(float& key, int& at) {
    const float top = max_over_warp(key);
    at = __reduce_min_sync(0xffffffffu, key == top ? at : 0x7fffffff);
    key = top;
}
// A barrier of the cluster's CTAs that orders nothing in memory.
__device__ inline void cluster_meet() {
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ inline float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T> __global__ void __launch_bounds__(kThr + 32, 1) verify_walk(const VerifyCall a) {
    extern __shared__ uint4 slots[];
    __shared__ Stats in_stats[2][kMaxCluster * kWarps];
    __shared__ Pick in_picks[2][kMaxCluster * kWarps];
    __shared__ uint64_t arrived[2], row_full[2], noise_full;
    __shared__ Order orders[2];
    __shared__ int parents[kMaxDrafts], tokens[kMaxDrafts], removed[kMaxDrafts];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int s = int(blockIdx.x) / C;
    const int r0 = a.cu_lens[s], r1 = a.cu_lens[s + 1], rows = r1 - r0;
    if (bad_rows(r0, r1, a.total_rows, a.max_rows) || rows == 0) {  // the whole cluster
        if (rank == 0 && tid == 0) {
            if (bad_rows(r0, r1, a.total_rows, a.max_rows)) flag(a.dev_status, PA_DEV_BAD_LEN);
            a.accepted_cu[s + 1] = 0;
            a.next_tokens[s] = -1;
        }
        return;
    }
    const float heat = a.temperature[s];  // not there where there are no rows at all
    const int V = a.vocab;
    const bool greedy = !(heat > 0.f);
    // neither infinite nor 0: a difference of 0 stays 0, one of -infinity stays that
    const float c = greedy ? kLog2e : fmaxf(fminf(kLog2e / heat, 3.402823466e38f), 1.175494351e-38f);
    const bool draft = !greedy && a.draft;
    const float* const noise = a.noise + int64_t(s) * V;

    // A row: single elements up to the first 16-byte boundary, units of eight, a
    // run of them to a CTA, single elements.
    struct Row {
        const T* p;
        const T* q;  // the draft's, or nullptr
        int head;    // single elements before the units
    };
    auto row_at = [&](int t, bool with_q) {
        Row r;
        r.p = static_cast<const T*>(a.logits) + int64_t(r0 + t) * a.logits_stride;
        r.q = with_q && draft ? static_cast<const T*>(a.draft) + int64_t(r0 + t) * a.draft_stride : nullptr;
        r.head = min(V, int((16 - (reinterpret_cast<uintptr_t>(r.p) & 15)) & 15) / int(sizeof(T)));
        return r;
    };
    // the CTA's first unit and the number of its units
    struct Span {
        int first, count;
    };
    auto run_of = [&](int head) {
        const int64_t units = (V - head) >> 3;
        const int first = int(units * rank / C);
        return Span{first, int(units * (rank + 1) / C) - first};
    };
    const int noise_head = row_at(0, false).head;
    const int most = ((V >> 3) + C - 1) / C + 1;  // units of a CTA at most
    constexpr int kAll = int(kRoom / 16), kFour = 4 * kParts<T>;
    const bool noise_staged = !greedy && wide_at(noise + noise_head) && most <= kAll / (kFour + 2);
    const int room = kAll / (noise_staged ? kFour + 2 : kFour);  // units of a row
    auto slot_of = [&](int held, int which, int unit) { return slots + ((2 * held + which) * room + unit) * kParts<T>; };
    uint4* const noise_slots = slots + room * kFour;
    for (int t = tid; t < rows; t += kThr + 32) {
        const int p = t ? a.parents[r0 + t] : -1, token = t ? a.tokens[r0 + t] : -1;
        const bool good = t && p >= 0 && p < t && token >= 0 && token < V;
        if (t && !good && rank == 0) flag(a.dev_status, PA_DEV_BAD_INDEX);
        parents[t] = good ? p : -1;  // nobody's child
        tokens[t] = token;
    }
    const uint32_t bytes = uint32_t(C) * kWarps * (sizeof(Stats) + sizeof(Pick));  // of an exchange
    // a row's first units, its draft's, to the slots of `held`, what is beyond them to L2 (one thread)
    auto copy_row = [&](int t, bool with_q, int held) {
        const Row r = row_at(t, with_q);
        const Span run = run_of(r.head);
        const uint32_t n = uint32_t(min(run.count, room)) * (8 * sizeof(T)), beyond = uint32_t(run.count) * (8 * sizeof(T)) - n;
        const T* p = r.p + r.head + 8 * run.first;
        const T* q = r.q && wide_at(r.q + r.head) ? r.q + r.head + 8 * run.first : nullptr;
        mbar_arrive_expect_tx(&row_full[held], q ? 2 * n : n);
        if (n) copy_bulk(slot_of(held, 0, 0), p, n, &row_full[held]);
        if (n && q) copy_bulk(slot_of(held, 1, 0), q, n, &row_full[held]);
        if (beyond) prefetch_bulk(p + 8 * room, beyond);
        if (beyond && q) prefetch_bulk(q + 8 * room, beyond);
    };
    if (tid == kThr) {  // the leader's first lane
        for (int i = 0; i < 2; ++i) {
            mbar_init(&arrived[i], 1);
            mbar_init(&row_full[i], 1);
        }
        mbar_init(&noise_full, 1);
        mbar_fence_init();
        for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&arrived[i], bytes);
        fence_proxy_async_smem();
        copy_row(0, rows > 1, 0);  // the draft's before it is known whether the row has children
        const Span run = run_of(noise_head);
        const uint32_t n = noise_staged ? uint32_t(run.count) * 32u : 0u;
        mbar_arrive_expect_tx(&noise_full, n);
        const float* from = noise + noise_head + 8 * run.first;
        if (n) copy_bulk(noise_slots, from, n, &noise_full);
        if (!greedy && !noise_staged && run.count > 1) {  // to L2, between the boundaries in it
            const char* p = reinterpret_cast<const char*>((reinterpret_cast<uintptr_t>(from) + 15) & ~uintptr_t(15));
            prefetch_bulk(p, uint32_t(reinterpret_cast<const char*>(from + 8 * run.count) - p) & ~15u);
        }
    }
    cluster.sync();  // the barriers are there before anyone sends

    // children of `here` among rows base .. base + 31, or the next such run that has some
    auto window = [&](int here, int& base) -> unsigned {
        for (; base < rows; base += 32) {
            const unsigned m = __ballot_sync(0xffffffffu, base + lane < rows && parents[base + lane] == here);
            if (m) return m;
        }
        return 0u;
    };

    int turn = 0;  // exchanges so far

    if (warp == kWarps) {
        // ================================ leader ================================
        bool lost = false;  // an exchange gave up
        const uint64_t limit = a.debug_timeout ? kTestNs : kWaitNs;
        // the cluster's results of an exchange
        auto wait = [&] {
            const int at = turn & 1;
            // testing: the first CTA gives up on its first exchange, the others go on
            const bool now = a.debug_timeout && rank == 0 && turn == 0;
            if (now || !__all_sync(0xffffffffu, mbar_wait_ns(&arrived[at], (turn >> 1) & 1, limit))) {
                lost = true;
                return at;
            }
            if (lane == 0) mbar_arrive_expect_tx(&arrived[at], bytes);  // for the exchange after the next
            ++turn;
            return at;
        };
        int ordered = 0;
        auto order = [&](const Order& o) {
            if (lane == 0) orders[ordered & 1] = o;
            ++ordered;
            __syncthreads();
        };
        const int n = C * kWarps;
        int here = 0, count = 0, next = -1;
        int held = 0, fills[2] = {1, 0};  // the row at hand; copies to the slots so far
        auto fill = [&](int t, bool with_q, int to) {
            if (lane == 0) {
                fence_proxy_async_smem();  // behind what the passes did there, by way of the last order
                copy_row(t, with_q, to);
            }
            ++fills[to];
        };
        for (;;) {
            if (rank == 0 && lane == 0) a.accepted[r0 + count] = r0 + here;
            ++count;
            int base = here + 1;
            unsigned children = window(here, base);
            const Row row = row_at(here, children != 0);
            // the row that the walk most likely goes on to
            const int guess = children ? base + __ffs(children) - 1 : -1;
            if (guess >= 0) {
                int after = guess + 1;
                fill(guess, window(guess, after) != 0, held ^ 1);
            }
            // the lane's child: its logits and its random number
            T x_mine = T(0.f), y_mine = T(0.f);
            float u_mine = 0.f;
            auto look = [&] {
                if ((children >> lane) & 1u) {
                    const int token = tokens[base + lane];
                    u_mine = a.uniform[r0 + base + lane];
                    x_mine = row.p[token];
                    if (row.q) y_mine = row.q[token];
                }
            };
            look();
            // the row's largest logit and sum, the draft's: the largest values first, then every sum once
            const int at = wait();
            if (lost) break;
            constexpr int kMine = kMaxCluster * kWarps / 32;
            Stats o[kMine];
            Stat P = {-INFINITY, 0.f}, Q = {-INFINITY, 0.f};
#pragma unroll
            for (int j = 0; j < kMine; ++j)
                if (lane + 32 * j < n) o[j] = in_stats[at][lane + 32 * j];
#pragma unroll
            for (int j = 0; j < kMine; ++j)
                if (lane + 32 * j < n) P.top = fmaxf(P.top, o[j].p.top), Q.top = fmaxf(Q.top, o[j].q.top);
            P.top = max_over_warp(P.top);
            Q.top = max_over_warp(Q.top);
#pragma unroll
            for (int j = 0; j < kMine; ++j)
                if (lane + 32 * j < n) P.sum += sum_at(o[j].p, P.top, c), Q.sum += sum_at(o[j].q, Q.top, c);
            P.sum = warp_sum(P.sum);
            Q.sum = warp_sum(Q.sum);
            int top_at = V;
            if (greedy) {
                float key = -INFINITY;
                for (int i = lane; i < n; i += 32) better(key, top_at, in_picks[at][i].key, in_picks[at][i].at);
                better_over_warp(key, top_at);
            }
            if (!usable(P) || (row.q && !usable(Q))) {
                if (rank == 0 && lane == 0) flag(a.dev_status, PA_DEV_BAD_VALUE);
                break;
            }
            // what is left of p is max(p - used q, 0) / mass
            const float p_of = rcp(P.sum), q_of = row.q ? rcp(Q.sum) : 0.f;
            // `used` of q in exponentials of the target's scale; 1 where the sums are equal (a division: 43.4 us
            // for 16 trees instead of 43.0)
            const float ratio = P.sum == Q.sum ? 1.f : P.sum * q_of;
            float used = 0.f, mass = 1.f, kept = -1.f;  // kept: what `used` was before the last child's rejection
            int dropped = 0;                            // certain drafts rejected here
            int went = 0;
            while (children) {
                const int l = __ffs(children) - 1, t = base + l;
                const float x = __shfl_sync(0xffffffffu, Elt<T>::f(x_mine), l);
                const float y = __shfl_sync(0xffffffffu, Elt<T>::f(y_mine), l);
                const float u = __shfl_sync(0xffffffffu, u_mine, l);
                const int token = tokens[t];
                bool again = false;
                float p = 0.f;
                if (greedy) {
                    if (token == top_at) went = t;
                } else {
                    const float ex = ex2((x - P.top) * c);
                    float q = 1.f;
                    p = ex * p_of;
                    if (row.q) {
                        const float ey = ex2((y - Q.top) * c);
                        q = ey * q_of;
                        p = left_of(ex, ey, used * ratio) * p_of * rcp(mass);
                    } else {
                        for (int i = lane; i < dropped; i += 32) again |= removed[i] == token;
                        again = __any_sync(0xffffffffu, again);
                        p = again ? 0.f : p * rcp(mass);
                    }
                    if (p > 0.f && u * q < p) went = t;
                }
                if (went) break;
                children &= children - 1;
                if (!children) {
                    base += 32;
                    children = window(here, base);
                    if (children) look();
                }
                if (greedy) continue;
                if (!row.q) {
                    if (!again && mass - p * mass > 0.f) {
                        mass -= p * mass;
                        if (lane == 0) removed[dropped] = token;
                        __syncwarp();
                        ++dropped;
                    }
                } else if (!children) {
                    kept = used;
                    used += mass;
                } else {
                    const float more = used + mass;
                    order(Order{kMass, 0, 0, 0, P.top, Q.top, more * ratio});
                    const int from = wait();
                    if (lost) break;
                    float sum = 0.f;
                    for (int i = lane; i < n; i += 32) sum += in_picks[from][i].key;
                    sum = warp_sum(sum) * p_of;
                    if (sum > 0.f) {
                        used = more;
                        mass = sum;
                    }
                }
            }
            if (lost) break;
            if (went) {
                held ^= 1;
                if (went != guess) {  // behind the guess's copies to the same slots
                    if (!__all_sync(0xffffffffu, mbar_wait_ns(&row_full[held], (fills[held] - 1) & 1, kWaitNs))) {
                        lost = true;
                        break;
                    }
                    int after = went + 1;
                    fill(went, window(went, after) != 0, held);
                }
                order(Order{kGo, went, (fills[held] - 1) & 1, 0, 0.f, 0.f, 0.f});
                here = went;
                continue;
            }
            if (greedy) {
                next = top_at;
                break;
            }
            for (;;) {
                order(Order{kPick, 0, 0, dropped, P.top, Q.top, used * ratio});
                const int from = wait();
                if (lost) break;
                float key = 0.f;
                int where = V;
                for (int i = lane; i < n; i += 32) better(key, where, in_picks[from][i].key, in_picks[from][i].at);
                better_over_warp(key, where);
                if (key > 0.f) {
                    next = where;
                    break;
                }
                if (kept < 0.f) {
                    if (rank == 0 && lane == 0) flag(a.dev_status, PA_DEV_BAD_VALUE);
                    break;
                }
                used = kept;  // nothing was left behind the last rejection: p is as it was
                kept = -1.f;
            }
            break;
        }
        order(Order{kStop, 0, 0, 0, 0.f, 0.f, 0.f});
        // nobody leaves with copies under way
        for (int i = 0; i < 2; ++i)
            if (fills[i]) mbar_wait_ns(&row_full[i], (fills[i] - 1) & 1, kWaitNs);
        mbar_wait_ns(&noise_full, 0, kWaitNs);
        if (rank == 0 && lane == 0) {
            if (lost) flag(a.dev_status, PA_DEV_TIMEOUT);
            a.accepted_cu[s + 1] = count;
            a.next_tokens[s] = next;
        }
        __syncwarp();
        // Others may be an exchange ahead of a CTA that gave up, and send to its shared
        // memory: it stays until all of them have stopped and what they sent is there.
        // (Who did not give up has waited for all that is sent to it.)
        cluster_meet();
        if (lost)
            for (int i = 0; i < 2; ++i) mbar_wait_ns(&arrived[(turn + i) & 1], ((turn + i) >> 1) & 1, kDrainNs);
        return;
    }

    // ================================== passes ==================================
    // Sends the warp's result to every CTA of the cluster.  A place is written
    // again by the exchange after the next, which nobody begins before its leader
    // has read the next, for which all have sent.
    auto send = [&](const Stats& stats, const Pick& pick) {
        const int at = turn++ & 1;
        if (lane < C) {
            const uint32_t bar = in_cta(smem_u32(&arrived[at]), lane);
            send16(in_cta(smem_u32(&in_stats[at][rank * kWarps + warp]), lane), bar, *reinterpret_cast<const uint4*>(&stats));
            send16(in_cta(smem_u32(&in_picks[at][rank * kWarps + warp]), lane), bar, *reinterpret_cast<const uint4*>(&pick));
        }
    };
    int taken = 0;
    auto next_order = [&]() -> const Order* {
        __syncthreads();
        return &orders[taken++ & 1];
    };
    int here = 0, held = 0, phase = 0;  // the row at hand, its slots and the phase of the copies to them
    bool again_from_start = false;
    // body(first index of a round, units, row) for rounds of `room` of the CTA's
    // units.  The next round's come to the slots when one is done with, and the
    // first one's back before the next pass over the row.
    auto rounds = [&](const Row& row, auto&& body) {
        const Span run = run_of(row.head);
        const bool more = run.count > room;
        auto stage_round = [&](int c0) {
            for (int u = tid; u < room && c0 + u < run.count; u += kThr) {
                const int at = row.head + 8 * (run.first + c0 + u);
                stage8<T>(slot_of(held, 0, u), row.p + at);
                if (row.q) stage8<T>(slot_of(held, 1, u), row.q + at);
            }
            cp_commit();
        };
        if (more && again_from_start) stage_round(0);
        for (int c0 = 0; c0 < run.count; c0 += room) {
            cp_wait<0>();
            body(row.head + 8 * (run.first + c0), min(room, run.count - c0));
            if (more) stage_round(c0 + room);
        }
        again_from_start = true;
    };
    // the thread's element outside the units, or -1
    auto single_of = [&](int head) {
        const int behind = head + ((V - head) >> 3 << 3);
        return rank == C - 1 && tid < head + V - behind ? (tid < head ? tid : behind + tid - head) : -1;
    };
    bool with_draft;
    {
        int base = 1;
        with_draft = draft && window(0, base);  // nothing is used of a row without children
    }
    bool fine = true;
    for (;;) {
        const Row row = row_at(here, with_draft);
        const int single = single_of(row.head);
        float one_p = 0.f, one_q = 0.f;
        if (single >= 0) {
            one_p = Elt<T>::f(row.p[single]);
            if (row.q) one_q = Elt<T>::f(row.q[single]);
        }
        if (row.q && !wide_at(row.q + row.head)) {  // no bulk copy takes it
            const Span run = run_of(row.head);
            for (int u = tid; u < room && u < run.count; u += kThr)
                stage8<T>(slot_of(held, 1, u), row.q + row.head + 8 * (run.first + u));
            cp_commit();
        }
        fine &= __all_sync(0xffffffffu, mbar_wait_ns(&row_full[held], phase, kWaitNs));
        again_from_start = false;
        Run run_p = {-INFINITY, 0}, run_q = {-INFINITY, 0};
        Pick pick = {-INFINITY, V, {0, 0}};
        auto first_place = [&](float x, int at) {  // greedy: a thread meets indices in ascending order but for the ends
            if (x > pick.key || (x == pick.key && at < pick.at)) pick.key = x, pick.at = at;
        };
        rounds(row, [&](int at, int units) {
            // the largest values first, then all exponentials against them
            float top_p = -INFINITY, top_q = -INFINITY;
#pragma unroll 4
            for (int u = tid; u < units; u += kThr) {
                top_p = fmaxf(top_p, max_slot<T>(slot_of(held, 0, u)));
                if (with_draft) top_q = fmaxf(top_q, max_slot<T>(slot_of(held, 1, u)));
            }
            const float ref_p = raise(run_p, top_p, c), ref_q = raise(run_q, top_q, c);
#pragma unroll 2
            for (int u = tid; u < units; u += kThr) {
                float x[8];
                take_slot<T>(slot_of(held, 0, u), x);
                add8(run_p, x, ref_p, c);
                if (greedy) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) first_place(x[e], at + 8 * u + e);
                }
                if (with_draft) {
                    take_slot<T>(slot_of(held, 1, u), x);
                    add8(run_q, x, ref_q, c);
                }
            }
        });
        if (single >= 0) {
            take1(run_p, one_p, c);
            if (with_draft) take1(run_q, one_q, c);
            if (greedy) first_place(one_p, single);
        }
        Stats stats = {over_warp(run_p, c), {-INFINITY, 0.f}};
        if (with_draft) stats.q = over_warp(run_q, c);
        if (greedy) better_over_warp(pick.key, pick.at);
        send(stats, pick);
        const Order* o = next_order();
        while (o->what == kMass || o->what == kPick) {
            // what is left of p times P.sum, of which a draft's exponential takes `less`
            const float p_top = o->p_top, q_top = o->q_top, less = o->less;
            auto left = [&](float x, float y) {
                const float p = ex2((x - p_top) * c);
                return less > 0.f ? left_of(p, ex2((y - q_top) * c), less) : p;
            };
            if (o->what == kMass) {
                float sum = 0.f;
                rounds(row, [&](int, int units) {
#pragma unroll 2
                    for (int u = tid; u < units; u += kThr) {
                        float x8[8], y8[8];
                        take_slot<T>(slot_of(held, 0, u), x8);
                        take_slot<T>(slot_of(held, 1, u), y8);
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum += left(x8[e], y8[e]);
                    }
                });
                if (single >= 0) sum += left(one_p, one_q);
                pick.key = warp_sum(sum);
            } else {
                const bool wide = wide_at(noise + row.head), staged = noise_staged && noise_head == row.head;
                if (staged) fine &= __all_sync(0xffffffffu, mbar_wait_ns(&noise_full, 0, kWaitNs));
                float best = 0.f;
                int best_at = V;
                // rejected certain drafts among the n places from `at`, a bit each
                auto out_of = [&](int at, unsigned n) {
                    unsigned bits = 0;
                    for (int k = 0; k < o->dropped; ++k) {
                        const unsigned d = unsigned(removed[k] - at);
                        if (d < n) bits |= 1u << d;
                    }
                    return bits;
                };
                auto weigh = [&](float p, float e, int at, bool out) {
                    const float key = p * rcp(e);  // a NaN is never better, nor a number below 0
                    if (!out && (key > best || (key == best && key > 0.f && at < best_at))) {
                        best = key;
                        best_at = at;
                    }
                };
                rounds(row, [&](int at0, int units) {
#pragma unroll 1
                    for (int u = tid; u < units; u += kThr) {
                        const int at = at0 + 8 * u;
                        float x8[8], y8[8], e8[8];
                        take_slot<T>(slot_of(held, 0, u), x8);
                        if (row.q) take_slot<T>(slot_of(held, 1, u), y8);
                        if (staged)
                            take_slot<float>(noise_slots + 2 * u, e8);
                        else if (wide)
                            take_slot<float>(reinterpret_cast<const uint4*>(noise + at), e8);
                        else
                            read8(noise + at, a.noise, a.noise + int64_t(a.num_seqs) * V, e8);
                        const unsigned out = out_of(at, 8);
#pragma unroll
                        for (int e = 0; e < 8; ++e) weigh(left(x8[e], y8[e]), e8[e], at + e, (out >> e) & 1u);
                    }
                });
                if (single >= 0) weigh(left(one_p, one_q), noise[single], single, out_of(single, 1));
                better_over_warp(best, best_at);
                pick.key = best;
                pick.at = best_at;
            }
            send(stats, pick);
            o = next_order();
        }
        if (o->what == kStop) break;
        here = o->went;
        phase = o->phase;
        held ^= 1;
        int after = here + 1;
        with_draft = draft && window(here, after);
    }
    cp_wait<0>();  // nobody leaves with copies under way
    if (!fine) flag(a.dev_status, PA_DEV_TIMEOUT);
    __syncwarp();
    cluster_meet();  // see the leader's
}

// Joins the sequences' lists: the walk left counts in accepted_cu and each
// list at its sequence's own rows, which lie at or behind its place in the
// joined one, so a tile of places can be read, then written, in ascending order:
// the sequences of a round (one a thread), then the next ones'.
__global__ void __launch_bounds__(kPackThr) verify_pack(const VerifyCall a) {
    __shared__ int sums[kPackThr / 32];
    __shared__ int ends[kPackThr], starts[kPackThr];  // in the joined list; a sequence's own rows
    pdl_wait_primary();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    if (tid == 0) a.accepted_cu[0] = 0;
    for (int s0 = 0; s0 < a.num_seqs; s0 += kPackThr) {
        const int s = s0 + tid;
        const int n = s < a.num_seqs ? a.accepted_cu[s + 1] : 0;
        const int start = s < a.num_seqs ? a.cu_lens[s] : 0;
        int v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < kPackThr / 32; ++w) {
            if (w < warp) v += sums[w];
            all += sums[w];
        }
        ends[tid] = base + v;
        starts[tid] = start;
        if (s < a.num_seqs) {
            a.accepted_cu[s + 1] = base + v;
            if (a.new_lens) a.new_lens[s] = a.context_lens[s] + n;
        }
        __syncthreads();
        const int stop = min(base + all, a.total_rows);
        for (int j0 = base; j0 < stop; j0 += kPackThr) {
            const int j = j0 + tid;
            int row = -1;
            if (j < stop) {
                int lo = 0, hi = kPackThr - 1;  // the first sequence that ends behind j
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (ends[mid] > j)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                row = a.accepted[starts[lo] + j - (lo ? ends[lo - 1] : base)];
            }
            __syncthreads();
            if (j < stop) a.accepted[j] = row;
            __syncthreads();
        }
        base += all;
    }
    for (int j = base + tid; j < a.total_rows; j += kPackThr) a.accepted[j] = -1;
}

template <typename T> cudaError_t launch_walk(const VerifyCall& c, cudaStream_t st) {
    static std::atomic<uint64_t> wide{0}, allowed{0};
    const void* kern = reinterpret_cast<const void*>(verify_walk<T>);
    cudaError_t e = allow_wide_clusters(kern, wide);
    if (e == cudaSuccess) e = allow_shared_memory(kern, kRoom, allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThr + 32);
    cfg.dynamicSmemBytes = kRoom;
    cfg.stream = st;
    // As wide a cluster as there is at once for every sequence, each CTA with a unit
    // for every second thread of its passes (one sequence, 16000 tokens: 4 CTAs 20.2 us,
    // 2 22.2, 8 21.8).  A cluster lies in one group of SMs, so that the GPU holds 7 of 16
    // CTAs, 15 of 8, 23 of 6, 28 of 5, 36 of 4, 46 of 3, 76 of 2, and behind the last
    // one a sequence waits: chains of 5, 131072 tokens, 8 sequences 35 us with 16 CTAs
    // each, 27 with 8; 18 45 us with 8, 31 with 6; 26 46 with 6, 38 with 5; 38 62 with 4,
    // 54 with 3.  Of 8 two more run at once than the 15 that CUDA's query counts where all
    // 152 SMs are there: 17 chains 27.5 us, with 6 CTAs each 31; 16 trees 37, with 6 45.
    // Any other answer is taken as it is, 0 where the query fails.
    static std::atomic<uint16_t> known[64][17];
    constexpr int kSizes[] = {kMaxCluster, 8, 6, 5, 4, 3, 2, 1};
    auto fits = [&](int size) {
        if ((c.vocab / 8 << 1) < kThr * size) return false;
        const int n = clusters_at_once(kern, cfg, size, known);
        return c.num_seqs <= (size == 8 && n == 15 ? 17 : n);
    };
    int pick = 0;
    while (kSizes[pick] > 1 && !fits(kSizes[pick])) ++pick;
    const int size = kSizes[pick];
    cfg.gridDim = dim3(unsigned(c.num_seqs) * size);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_walk<T>, c);
}

}  // namespace

cudaError_t launch_verify(const VerifyCall& c, cudaStream_t st) {
    const cudaError_t e = c.dtype == PA_F32   ? launch_walk<float>(c, st)
                          : c.dtype == PA_F16 ? launch_walk<__half>(c, st)
                                              : launch_walk<__nv_bfloat16>(c, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(verify_pack, dim3(1), dim3(kPackThr), 0, st, c);
}

}  // namespace pa
