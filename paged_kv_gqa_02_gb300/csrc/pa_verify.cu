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
// largest p_i / e_i for exponential e_i: a comparison of single terms, which
// rounding can turn only where two are within a few units of 2^-24 of each
// other, while a search in running sums would meet a border every few 2^-24 in a
// vocabulary's tail.  M does not matter to it.
//
// The walk's time is a chain of passes, each bound by latency: the exponentials
// of a row and one exchange.  A thread's part of the rows waits in slots of
// shared memory that only it uses: the row at hand, for all of its passes, and
// the first child's, on its way while the parent's is decided; the random numbers
// from the start.  For an exchange every warp sends its result to the shared
// memory of every CTA of the cluster, counted by an mbarrier there.  A warp of
// its own, the leader, reads what it needs of the children meanwhile, joins the
// results and orders the next pass; leaders of a cluster join the same in the same
// order and so decide the same.  Only rank 0 writes.  A second kernel joins the
// sequences' lists.
#include <cooperative_groups.h>

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
constexpr int kSingles = 16;      // elements of a row outside its units of eight at most, and two
constexpr int kPackThr = 1024;
constexpr uint64_t kWaitNs = 2000000000ull;  // an exchange gives up after 2 s

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
    int what, went;
    int dropped;              // certain drafts rejected
    float p_top, q_top, less; // what is left: 2^((x - p_top) c) - less 2^((y - q_top) c), not below 0
};
// A thread's running Stat, the sum in two parts.
struct Run {
    float top;
    uint64_t sum;
};

// Whether p lies on a 16-byte boundary.
template <typename T> __device__ inline bool wide_at(const T* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

__device__ inline void cp_async16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ inline void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ inline void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Slots of shared memory for units of eight elements: a thread's k-th unit of a
// row, its 16-byte parts kThr apart.
template <typename T> struct Stage {
    static constexpr int kParts = 8 / Elt<T>::kVec;
    static constexpr int kSlots = 4 / kParts;                    // a thread's units of a row
    static constexpr int kRow = kSlots * kParts * kThr;          // 16-byte parts of a row
    static constexpr int kNoise = kSlots * 2 * kThr;
    static constexpr size_t kBytes = size_t(4 * kRow + kNoise) * 16;  // two rows and their drafts', random numbers
};
__device__ inline void cp_async4(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

// Eight elements to the thread's slot and from it.  Copies that arrive later,
// but for 16-bit elements off the 16-byte boundaries.
template <typename T> __device__ inline void stage8(uint4* slot, const T* p) {
    if (wide_at(p)) {
#pragma unroll
        for (int i = 0; i < 8 / Elt<T>::kVec; ++i)
            cp_async16(smem_u32(slot + i * kThr), reinterpret_cast<const uint4*>(p) + i);
    } else if (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) cp_async4(smem_u32(slot + i / 4 * kThr) + 4 * (i % 4), p + i);
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
    for (int i = 0; i < 8 / Elt<T>::kVec; ++i) vec_to_f32<T>(slot[i * kThr], x + i * Elt<T>::kVec);
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
__device__ inline void take8(Run& s, const float (&x)[8], float c) {
    const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    const float ref = raise(s, top, c);
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
__device__ inline float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T> __global__ void __launch_bounds__(kThr + 32, 1) verify_walk(const VerifyCall a) {
    extern __shared__ uint4 slots[];
    __shared__ Stats in_stats[2][kMaxCluster * kWarps];
    __shared__ Pick in_picks[2][kMaxCluster * kWarps];
    __shared__ uint64_t arrived[2];
    __shared__ Order orders[2];
    __shared__ float singles[2][2][kSingles];
    __shared__ int parents[kMaxDrafts], tokens[kMaxDrafts], removed[kMaxDrafts];
    using St = Stage<T>;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int s = int(blockIdx.x) / C;
    const int r0 = a.cu_lens[s], r1 = a.cu_lens[s + 1], rows = r1 - r0;
    const float heat = a.temperature[s];
    if (bad_rows(r0, r1, a.total_rows, a.max_rows) || rows == 0) {  // the whole cluster
        if (rank == 0 && tid == 0) {
            if (bad_rows(r0, r1, a.total_rows, a.max_rows)) flag(a.dev_status, PA_DEV_BAD_LEN);
            a.accepted_cu[s + 1] = 0;
            a.next_tokens[s] = -1;
        }
        return;
    }
    const int V = a.vocab;
    const bool greedy = !(heat > 0.f);
    const float c = greedy ? kLog2e : fminf(kLog2e / heat, 3.402823466e38f);
    const float* const noise = a.noise + int64_t(s) * V;
    const int worker = rank * kThr + tid, workers = C * kThr;

    // A row as the threads read it: single elements up to the first 16-byte
    // boundary, units of eight, the cluster's threads in turn, single elements.
    struct Row {
        const T* p;
        const T* q;  // the draft's, or nullptr
        int head;    // single elements before the units
    };
    auto row_at = [&](int t, bool with_q) {
        Row r;
        r.p = static_cast<const T*>(a.logits) + int64_t(r0 + t) * a.logits_stride;
        r.q = with_q && !greedy && a.draft ? static_cast<const T*>(a.draft) + int64_t(r0 + t) * a.draft_stride : nullptr;
        r.head = min(V, int((16 - (reinterpret_cast<uintptr_t>(r.p) & 15)) & 15) / int(sizeof(T)));
        return r;
    };
    auto units_of = [&](int head) { return (V - head) >> 3; };
    // the thread's single element, or -1
    auto single_of = [&](int head) {
        const int behind = head + 8 * units_of(head);
        return rank == C - 1 && tid < head + V - behind ? (tid < head ? tid : behind + tid - head) : -1;
    };
    uint4* const noise_slots = slots + 4 * St::kRow + tid;
    auto slot_of = [&](int held, int draft, int k) { return slots + (2 * held + draft) * St::kRow + k * St::kParts * kThr + tid; };
    // the first units of a row and of its draft's on their way to the slots of `held`
    auto fetch = [&](const Row& r, int held) {
        const int units = units_of(r.head), single = single_of(r.head);
#pragma unroll
        for (int k = 0; k < St::kSlots; ++k) {
            const int i = worker + k * workers;
            if (i < units) {
                stage8<T>(slot_of(held, 0, k), r.p + r.head + 8 * i);
                if (r.q) stage8<T>(slot_of(held, 1, k), r.q + r.head + 8 * i);
            }
        }
        if (single >= 0) {
            singles[held][0][tid] = Elt<T>::f(r.p[single]);
            if (r.q) singles[held][1][tid] = Elt<T>::f(r.q[single]);
        }
        cp_commit();
    };
    // random numbers off the 16-byte boundaries are read where they lie
    auto noise_wide = [&](int head) { return wide_at(noise + head); };
    auto fetch_noise = [&](int head) {
        const int units = units_of(head);
        if (!noise_wide(head)) return;
#pragma unroll
        for (int k = 0; k < St::kSlots; ++k) {
            const int i = worker + k * workers;
            if (i < units) stage8<float>(noise_slots + 2 * k * kThr, noise + head + 8 * i);
        }
    };
    Row row = row_at(0, rows > 1);
    int held = 0;
    if (warp < kWarps) fetch(row, held);
    for (int t = tid; t < rows; t += kThr + 32) {
        const int p = t ? a.parents[r0 + t] : -1, token = t ? a.tokens[r0 + t] : -1;
        const bool good = t && p >= 0 && p < t && token >= 0 && token < V;
        if (t && !good && rank == 0) flag(a.dev_status, PA_DEV_BAD_INDEX);
        parents[t] = good ? p : -1;  // nobody's child
        tokens[t] = token;
    }
    const uint32_t bytes = uint32_t(C) * kWarps * (sizeof(Stats) + sizeof(Pick));  // of an exchange
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&arrived[i], 1);
            mbar_fence_init();
            mbar_arrive_expect_tx(&arrived[i], bytes);
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
        // the cluster's results of an exchange
        auto wait = [&] {
            const int at = turn & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_ns(&arrived[at], (turn >> 1) & 1, kWaitNs))) lost = true;
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
        for (;;) {
            if (rank == 0 && lane == 0) a.accepted[r0 + count] = r0 + here;
            ++count;
            int base = here + 1;
            unsigned children = window(here, base);
            row = row_at(here, children != 0);
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
                    p = ex2((x - P.top) * c) * p_of;
                    float q = 1.f;
                    if (row.q) {
                        q = ex2((y - Q.top) * c) * q_of;
                        p = fmaxf(p - used * q, 0.f) * rcp(mass);
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
                    order(Order{kMass, 0, 0, P.top, Q.top, more * q_of * P.sum});
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
                order(Order{kGo, went, 0, 0.f, 0.f, 0.f});
                here = went;
                continue;
            }
            if (greedy) {
                next = top_at;
                break;
            }
            for (;;) {
                order(Order{kPick, 0, dropped, P.top, Q.top, used * q_of * P.sum});
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
        order(Order{kStop, 0, 0, 0.f, 0.f, 0.f});
        if (rank == 0 && lane == 0) {
            if (lost) flag(a.dev_status, PA_DEV_TIMEOUT);
            a.accepted_cu[s + 1] = count;
            a.next_tokens[s] = next;
        }
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
    auto next_order = [&] {
        __syncthreads();
        return orders[taken++ & 1];
    };
    // f(eight of p, eight of q, first index, slot) over the thread's units of the row
    // at hand.  Units that have no slot of their own come to one that is done with,
    // and the first ones back to theirs before the next pass over the row.
    bool with_noise = false;  // the pass reads random numbers too
    bool again_from_start = false;
    auto over = [&](auto&& f) {
        const int units = units_of(row.head);
        const bool more = worker + St::kSlots * workers < units;
        auto stage_unit = [&](int slot, int i) {
            stage8<T>(slot_of(held, 0, slot), row.p + row.head + 8 * i);
            if (row.q) stage8<T>(slot_of(held, 1, slot), row.q + row.head + 8 * i);
            if (with_noise && noise_wide(row.head)) stage8<float>(noise_slots + 2 * slot * kThr, noise + row.head + 8 * i);
        };
        if (more && again_from_start) {
            cp_wait<0>();
#pragma unroll 1
            for (int k = 0; k < St::kSlots; ++k) stage_unit(k, worker + k * workers);
            cp_commit();
            cp_wait<0>();
        }
        int slot = 0;
#pragma unroll 1
        for (int i = worker; i < units; i += workers) {
            if (i >= St::kSlots * workers) cp_wait<St::kSlots - 1>();
            float x[8], y[8];
            take_slot<T>(slot_of(held, 0, slot), x);
            if (row.q) take_slot<T>(slot_of(held, 1, slot), y);
            f(x, y, row.head + 8 * i, slot);
            if (more) {
                if (i + St::kSlots * workers < units) stage_unit(slot, i + St::kSlots * workers);
                cp_commit();
            }
            slot = slot + 1 == St::kSlots ? 0 : slot + 1;
        }
        again_from_start = true;
    };
    int here = 0;
    {
        int base = 1;
        if (!window(0, base)) row.q = nullptr;  // nothing is used of a row without children
    }
    const int noise_head = row.head;
    if (!greedy) fetch_noise(row.head);
    cp_commit();
    bool first = true;
    for (;;) {
        if (first)
            cp_wait<1>();  // all but the random numbers
        else
            cp_wait<0>();
        first = false;
        again_from_start = false;
        Run run_p = {-INFINITY, 0}, run_q = {-INFINITY, 0};
        Pick pick = {-INFINITY, V, {0, 0}};
        auto first_place = [&](float x, int at) {  // greedy: a thread meets indices in ascending order but for the ends
            if (x > pick.key || (x == pick.key && at < pick.at)) pick.key = x, pick.at = at;
        };
        over([&](const float(&x)[8], const float(&y)[8], int at, int) {
            take8(run_p, x, c);
            if (row.q) take8(run_q, y, c);
            if (greedy) {
#pragma unroll
                for (int e = 0; e < 8; ++e) first_place(x[e], at + e);
            }
        });
        const int single = single_of(row.head);
        if (single >= 0) {
            take1(run_p, singles[held][0][tid], c);
            if (row.q) take1(run_q, singles[held][1][tid], c);
            if (greedy) first_place(singles[held][0][tid], single);
        }
        Stats stats = {over_warp(run_p, c), {-INFINITY, 0.f}};
        if (row.q) stats.q = over_warp(run_q, c);
        if (greedy) better_over_warp(pick.key, pick.at);
        send(stats, pick);
        // the row that the walk most likely goes on to
        int base = here + 1;
        const unsigned children = window(here, base);
        const int guess = children ? base + __ffs(children) - 1 : -1;
        Row ahead = {};
        if (guess >= 0) {
            int after = guess + 1;
            ahead = row_at(guess, window(guess, after) != 0);
            fetch(ahead, held ^ 1);
        }
        Order o = next_order();
        while (o.what == kMass || o.what == kPick) {
            // what is left of p times P.sum, of which a draft's exponential takes `less`
            auto left = [&](float x, float y) {
                const float p = ex2((x - o.p_top) * c);
                return o.less > 0.f ? fmaxf(p - ex2((y - o.q_top) * c) * o.less, 0.f) : p;
            };
            if (o.what == kMass) {
                float sum = 0.f;
                over([&](const float(&x8)[8], const float(&y8)[8], int, int) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum += left(x8[e], y8[e]);
                });
                if (single >= 0) sum += left(singles[held][0][tid], singles[held][1][tid]);
                pick.key = warp_sum(sum);
            } else {
                cp_wait<0>();
                if (!with_noise && noise_head != row.head) {  // another alignment than the first row's
                    fetch_noise(row.head);
                    cp_commit();
                    cp_wait<0>();
                }
                with_noise = true;
                float best = 0.f;
                int best_at = V;
                // rejected certain drafts among the n places from `at`, a bit each
                auto out_of = [&](int at, unsigned n) {
                    unsigned bits = 0;
                    for (int k = 0; k < o.dropped; ++k) {
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
                over([&](const float(&x8)[8], const float(&y8)[8], int at, int slot) {
                    float e8[8];
                    if (noise_wide(row.head))
                        take_slot<float>(noise_slots + 2 * slot * kThr, e8);
                    else
                        read8(noise + at, a.noise, a.noise + int64_t(a.num_seqs) * V, e8);
                    const unsigned out = out_of(at, 8);
#pragma unroll
                    for (int e = 0; e < 8; ++e) weigh(left(x8[e], y8[e]), e8[e], at + e, (out >> e) & 1u);
                });
                if (single >= 0)
                    weigh(left(singles[held][0][tid], singles[held][1][tid]), noise[single], single, out_of(single, 1));
                better_over_warp(best, best_at);
                pick.key = best;
                pick.at = best_at;
            }
            send(stats, pick);
            o = next_order();
        }
        if (o.what == kStop) break;
        here = o.went;
        if (here == guess) {
            row = ahead;
        } else {
            int after = here + 1;
            row = row_at(here, window(here, after) != 0);
            cp_wait<0>();  // the guess is still on its way there
            fetch(row, held ^ 1);
        }
        held ^= 1;
    }
    cp_wait<0>();  // nobody leaves with copies under way
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
    if (e == cudaSuccess) e = allow_shared_memory(kern, Stage<T>::kBytes, allowed);
    if (e != cudaSuccess) return e;
    // as many CTAs as the GPU holds at once, each with a unit for every thread
    int size = kMaxCluster;
    while (size > 1 && (int64_t(c.num_seqs) * size > 152 || c.vocab / 8 < size * kThr / 2)) size /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(c.num_seqs) * size);
    cfg.blockDim = dim3(kThr + 32);
    cfg.dynamicSmemBytes = Stage<T>::kBytes;
    cfg.stream = st;
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
