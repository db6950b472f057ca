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
// The walk's time is a chain of passes, each bound by latency: a read of the row
// (from L2: the first child's row and the random numbers are prefetched while
// earlier passes run), the exponentials, and one exchange.  For that, every warp
// sends its result to the shared memory of every CTA of the cluster, counted by
// an mbarrier there; each warp then joins all of them in the same order and takes
// the decisions itself.  Only rank 0 writes.  A second kernel joins the sequences'
// lists.
#include <cooperative_groups.h>

#include "pa_device.h"
#include "pa_pairs.cuh"
#include "pa_ptx.cuh"
#include "pa_rows.cuh"
#include "pa_serving.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kThr = 512;
constexpr int kWarps = kThr / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxDrafts = 1024;  // rows of a sequence
constexpr int kPackThr = 1024;
constexpr uint64_t kWaitNs = 2000000000ull;  // an exchange gives up after 2 s

// The largest logit and the sum of 2^((x - largest) c); with a NaN or an
// infinite largest one the sum is not finite.
struct Stat {
    float top, sum;
};
// What a warp found in a pass.
struct __align__(16) Slot {
    Stat p, q;
    float key;  // of the best candidate for the next token, or a sum
    int at;     // where the largest logit (greedy) or the best candidate is
    int pad[2];
};
// A thread's running Stat, the sum in two parts.
struct Run {
    float top;
    uint64_t sum;
};

// A row of the vocabulary as the threads read it: single elements up to the
// first 16-byte boundary, units of eight, single elements.
struct Span {
    int head, units;
};
template <typename T> __device__ inline Span span_of(const T* row, int vocab) {
    Span s;
    const int off = int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    s.head = min(vocab, off ? int(16 / sizeof(T)) - off : 0);
    s.units = (vocab - s.head) / 8;
    return s;
}
template <typename T> __device__ inline bool wide_at(const T* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Eight elements from p, by 16-byte loads where p is aligned.
template <typename T> struct Eight {
    uint4 v[8 / Elt<T>::kVec];
    __device__ inline void load(const T* p, bool wide) {
        if (wide) {
#pragma unroll
            for (int i = 0; i < 8 / Elt<T>::kVec; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
        } else {
            T* e = reinterpret_cast<T*>(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = __ldg(p + i);
        }
    }
    __device__ inline void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8 / Elt<T>::kVec; ++i) vec_to_f32<T>(v[i], x + i * Elt<T>::kVec);
    }
};

__device__ inline void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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

__device__ inline void raise(Run& s, float top, float c) {
    if (top > s.top) {
        const float down = ex2((s.top - top) * c);
        s.sum = pairs::mul(s.sum, pairs::pack(down, down));
        s.top = top;
    }
}
__device__ inline void take8(Run& s, const float (&x)[8], float c) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i]);
    raise(s, top, c);
    if (s.top > -INFINITY) {
        const uint64_t minus = pairs::pack(-s.top, -s.top), c2 = pairs::pack(c, c);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 e = pairs::unpack(pairs::mul(pairs::add(pairs::pack(x[i], x[i + 1]), minus), c2));
            s.sum = pairs::add(s.sum, pairs::pack(ex2(e.x), ex2(e.y)));
        }
    } else {  // a NaN is not lost
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (x[i] != x[i]) s.sum = pairs::pack(x[i], x[i]);
    }
}
__device__ inline void take1(Run& s, float x, float c) {
    raise(s, x, c);
    const float e = s.top > -INFINITY ? ex2((x - s.top) * c) : x != x ? x : 0.f;
    s.sum = pairs::add(s.sum, pairs::pack(e, 0.f));
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

template <typename T> __global__ void __launch_bounds__(kThr, 1) verify_walk(const VerifyCall a) {
    constexpr int kAhead = Elt<T>::kVec / 2;  // units of eight logits whose loads a thread has in flight
    __shared__ Slot inbox[2][kMaxCluster * kWarps];
    __shared__ uint64_t arrived[2];
    __shared__ int parents[kMaxDrafts], tokens[kMaxDrafts], removed[kMaxDrafts];
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
    const T* const logits = static_cast<const T*>(a.logits);
    const T* const draft = greedy ? nullptr : static_cast<const T*>(a.draft);
    const float* const noise = a.noise + int64_t(s) * V;
    const int worker = rank * kThr + tid, workers = C * kThr;
    // a line of 128 bytes to a thread
    auto prefetch = [&](const char* p, int64_t bytes) {
        for (int64_t i = int64_t(worker) * 128; i < bytes; i += int64_t(workers) * 128) prefetch_l2(p + i);
    };
    for (int t = tid; t < rows; t += kThr) {
        const int p = t ? a.parents[r0 + t] : -1, token = t ? a.tokens[r0 + t] : -1;
        const bool good = t && p >= 0 && p < t && token >= 0 && token < V;
        if (t && !good && rank == 0) flag(a.dev_status, PA_DEV_BAD_INDEX);
        parents[t] = good ? p : -1;  // nobody's child
        tokens[t] = token;
    }
    if (!greedy) prefetch(reinterpret_cast<const char*>(noise), int64_t(V) * sizeof(float));
    const uint32_t bytes = uint32_t(C) * kWarps * sizeof(Slot);  // of an exchange
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&arrived[i], 1);
            mbar_fence_init();
            mbar_arrive_expect_tx(&arrived[i], bytes);
        }
    }
    cluster.sync();  // the barriers are there before anyone sends

    int turn = 0;
    bool lost = false;  // an exchange gave up
    // Sends the warp's result to every CTA of the cluster and waits for all of
    // theirs; `meanwhile` runs in between.  A place is written again by the
    // exchange after the next, which nobody begins before all have sent for the
    // next, and so have read this one.
    auto exchange = [&](const Slot& mine, auto&& meanwhile) -> const Slot* {
        const int at = turn & 1;
        if (lane < C) {
            const uint32_t to = in_cta(smem_u32(&inbox[at][rank * kWarps + warp]), lane);
            const uint32_t bar = in_cta(smem_u32(&arrived[at]), lane);
            const uint4* v = reinterpret_cast<const uint4*>(&mine);
            send16(to, bar, v[0]);
            send16(to + 16, bar, v[1]);
        }
        meanwhile();
        if (!__all_sync(0xffffffffu, mbar_wait_ns(&arrived[at], (turn >> 1) & 1, kWaitNs))) lost = true;
        if (tid == 0) mbar_arrive_expect_tx(&arrived[at], bytes);  // for the exchange after the next
        ++turn;
        return inbox[at];
    };
    // f(index of eight) and g(index of one) over the row, the cluster's threads in turn
    auto over = [&](const Span& sp, auto&& f, auto&& g) {
        for (int i = worker; i < sp.units; i += kAhead * workers) f(i);
        const int behind = sp.head + 8 * sp.units, single = sp.head + (V - behind);
        if (rank == C - 1 && tid < single) g(tid < sp.head ? tid : behind + tid - sp.head);
    };
    // children of `here` among rows base .. base + 31, or the next such run that has some
    auto window = [&](int here, int& base) -> unsigned {
        for (; base < rows; base += 32) {
            const unsigned m = __ballot_sync(0xffffffffu, base + lane < rows && parents[base + lane] == here);
            if (m) return m;
        }
        return 0u;
    };

    int here = 0, count = 0, next = -1;
    for (;;) {
        if (rank == 0 && tid == 0) a.accepted[r0 + count] = r0 + here;
        ++count;
        const T* const row = logits + int64_t(r0 + here) * a.logits_stride;
        int base = here + 1;
        unsigned children = window(here, base);
        const T* const q_row = draft && children ? draft + int64_t(r0 + here) * a.draft_stride : nullptr;
        // the lane's child: its logits and its random number
        float x_mine = 0.f, y_mine = 0.f, u_mine = 0.f;
        auto look = [&] {
            if ((children >> lane) & 1u) {
                const int token = tokens[base + lane];
                u_mine = a.uniform[r0 + base + lane];
                x_mine = Elt<T>::f(row[token]);
                if (q_row) y_mine = Elt<T>::f(q_row[token]);
            }
        };
        look();
        const Span sp = span_of(row, V);
        const bool q_wide = q_row && wide_at(q_row + sp.head);
        Slot mine = {{-INFINITY, 0.f}, {-INFINITY, 0.f}, -INFINITY, V, {0, 0}};
        Run run_p = {-INFINITY, 0}, run_q = {-INFINITY, 0};
        auto first_place = [&](float x, int at) {  // greedy: a thread meets indices in ascending order but for the ends
            if (x > mine.key || (x == mine.key && at < mine.at)) mine.key = x, mine.at = at;
        };
        over(
            sp,
            [&](int i) {
                Eight<T> u[kAhead], v[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (i + k * workers < sp.units) {
                        const int at = sp.head + 8 * (i + k * workers);
                        u[k].load(row + at, true);
                        if (q_row) v[k].load(q_row + at, q_wide);
                    }
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (i + k * workers < sp.units) {
                        float x[8];
                        u[k].get(x);
                        take8(run_p, x, c);
                        if (greedy) {
                            const int at = sp.head + 8 * (i + k * workers);
#pragma unroll
                            for (int e = 0; e < 8; ++e) first_place(x[e], at + e);
                        }
                        if (q_row) {
                            v[k].get(x);
                            take8(run_q, x, c);
                        }
                    }
            },
            [&](int at) {
                const float x = Elt<T>::f(row[at]);
                take1(run_p, x, c);
                if (greedy) first_place(x, at);
                if (q_row) take1(run_q, Elt<T>::f(q_row[at]), c);
            });
        mine.p = over_warp(run_p, c);
        if (q_row) mine.q = over_warp(run_q, c);
        if (greedy) better_over_warp(mine.key, mine.at);
        const Slot* all = exchange(mine, [&] {  // the row that the walk most likely goes on to
            if (!children) return;
            const int t = base + __ffs(children) - 1;
            prefetch(reinterpret_cast<const char*>(logits + int64_t(r0 + t) * a.logits_stride), int64_t(V) * sizeof(T));
            if (draft && t + 1 < rows && parents[t + 1] == t)
                prefetch(reinterpret_cast<const char*>(draft + int64_t(r0 + t) * a.draft_stride), int64_t(V) * sizeof(T));
        });
        if (lost) break;
        // the cluster's: the largest values first, then every sum once
        Stat P = {-INFINITY, 0.f}, Q = {-INFINITY, 0.f};
        float top_key = -INFINITY;
        int top_at = V;
        for (int i = lane; i < C * kWarps; i += 32) {
            P.top = fmaxf(P.top, all[i].p.top);
            if (q_row) Q.top = fmaxf(Q.top, all[i].q.top);
            if (greedy) better(top_key, top_at, all[i].key, all[i].at);
        }
        P.top = max_over_warp(P.top);
        if (q_row) Q.top = max_over_warp(Q.top);
        if (greedy) better_over_warp(top_key, top_at);
        for (int i = lane; i < C * kWarps; i += 32) {
            P.sum += sum_at(all[i].p, P.top, c);
            if (q_row) Q.sum += sum_at(all[i].q, Q.top, c);
        }
        P.sum = warp_sum(P.sum);
        if (q_row) Q.sum = warp_sum(Q.sum);
        if (!usable(P) || (q_row && !usable(Q))) {
            if (rank == 0 && tid == 0) flag(a.dev_status, PA_DEV_BAD_VALUE);
            break;
        }
        // what is left of p is max(p - used q, 0) / mass
        const float p_of = 1.f / P.sum, q_of = q_row ? 1.f / Q.sum : 0.f;
        float used = 0.f, mass = 1.f, kept = -1.f;  // kept: what `used` was before the last child's rejection
        int dropped = 0;                            // certain drafts rejected here
        int went = 0;
        while (children) {
            const int l = __ffs(children) - 1, t = base + l;
            const float x = __shfl_sync(0xffffffffu, x_mine, l), y = __shfl_sync(0xffffffffu, y_mine, l);
            const float u = __shfl_sync(0xffffffffu, u_mine, l);
            const int token = tokens[t];
            bool again = false;
            float p = 0.f;
            if (greedy) {
                if (token == top_at) went = t;
            } else {
                p = ex2((x - P.top) * c) * p_of;
                float q = 1.f;
                if (q_row) {
                    q = ex2((y - Q.top) * c) * q_of;
                    p = fmaxf(p - used * q, 0.f) / mass;
                } else {
                    for (int i = lane; i < dropped; i += 32) again |= removed[i] == token;
                    again = __any_sync(0xffffffffu, again);
                    p = again ? 0.f : p / mass;
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
            if (!q_row) {
                if (!again && mass - p * mass > 0.f) {
                    mass -= p * mass;
                    __syncthreads();  // all warps have looked through the list
                    if (tid == 0) removed[dropped] = token;
                    ++dropped;
                    __syncthreads();
                }
            } else if (!children) {
                kept = used;
                used += mass;
            } else {
                const float more = used + mass, q_s = more * q_of;
                float sum = 0.f;
                auto rest = [&](float x, float y) {
                    sum += fmaxf(ex2((x - P.top) * c) * p_of - ex2((y - Q.top) * c) * q_s, 0.f);
                };
                over(
                    sp,
                    [&](int i) {
                        Eight<T> u[kAhead], v[kAhead];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k)
                            if (i + k * workers < sp.units) {
                                const int at = sp.head + 8 * (i + k * workers);
                                u[k].load(row + at, true);
                                v[k].load(q_row + at, q_wide);
                            }
#pragma unroll
                        for (int k = 0; k < kAhead; ++k)
                            if (i + k * workers < sp.units) {
                                float x8[8], y8[8];
                                u[k].get(x8);
                                v[k].get(y8);
#pragma unroll
                                for (int e = 0; e < 8; ++e) rest(x8[e], y8[e]);
                            }
                    },
                    [&](int at) { rest(Elt<T>::f(row[at]), Elt<T>::f(q_row[at])); });
                mine.key = warp_sum(sum);
                const Slot* sums = exchange(mine, [] {});
                if (lost) break;
                sum = 0.f;
                for (int i = lane; i < C * kWarps; i += 32) sum += sums[i].key;
                sum = warp_sum(sum);
                if (sum > 0.f) {
                    used = more;
                    mass = sum;
                }
            }
        }
        if (lost) break;
        if (went) {
            here = went;
            continue;
        }
        if (greedy) {
            next = top_at;
            break;
        }
        const bool e_wide = wide_at(noise + sp.head);
        for (;;) {
            // what is left of p times P.sum, and by how much the draft's exponentials count in it
            const float q_s = used * q_of * P.sum;
            float best = 0.f;
            int best_at = V;
            auto left = [&](float x, float y) {
                const float p = ex2((x - P.top) * c);
                return q_s > 0.f ? fmaxf(p - ex2((y - Q.top) * c) * q_s, 0.f) : p;
            };
            // rejected certain drafts among the n places from `at`, a bit each
            auto out_of = [&](int at, unsigned n) {
                unsigned bits = 0;
                for (int k = 0; k < dropped; ++k) {
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
            over(
                sp,
                [&](int i) {
                    Eight<T> u[kAhead], v[kAhead];
                    Eight<float> z[kAhead];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k)
                        if (i + k * workers < sp.units) {
                            const int at = sp.head + 8 * (i + k * workers);
                            u[k].load(row + at, true);
                            if (q_s > 0.f) v[k].load(q_row + at, q_wide);
                            z[k].load(noise + at, e_wide);
                        }
#pragma unroll
                    for (int k = 0; k < kAhead; ++k)
                        if (i + k * workers < sp.units) {
                            float x8[8], y8[8], e8[8];
                            u[k].get(x8);
                            if (q_s > 0.f) v[k].get(y8);
                            z[k].get(e8);
                            const int at = sp.head + 8 * (i + k * workers);
                            const unsigned out = out_of(at, 8);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                weigh(left(x8[e], q_s > 0.f ? y8[e] : 0.f), e8[e], at + e, (out >> e) & 1u);
                        }
                },
                [&](int at) {
                    weigh(left(Elt<T>::f(row[at]), q_s > 0.f ? Elt<T>::f(q_row[at]) : 0.f), noise[at], at, out_of(at, 1));
                });
            better_over_warp(best, best_at);
            mine.key = best;
            mine.at = best_at;
            const Slot* picks = exchange(mine, [] {});
            if (lost) break;
            best = 0.f;
            best_at = V;
            for (int i = lane; i < C * kWarps; i += 32) better(best, best_at, picks[i].key, picks[i].at);
            better_over_warp(best, best_at);
            if (best > 0.f) {
                next = best_at;
                break;
            }
            if (kept < 0.f) {
                if (rank == 0 && tid == 0) flag(a.dev_status, PA_DEV_BAD_VALUE);
                break;
            }
            used = kept;  // nothing was left behind the last rejection: p is as it was
            kept = -1.f;
        }
        break;
    }
    if (rank == 0 && tid == 0) {
        if (lost) flag(a.dev_status, PA_DEV_TIMEOUT);
        a.accepted_cu[s + 1] = count;
        a.next_tokens[s] = next;
    }
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
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_wide_clusters(reinterpret_cast<const void*>(verify_walk<T>), done);
    if (e != cudaSuccess) return e;
    // as many CTAs as the GPU holds at once, each with a unit for every thread
    int size = kMaxCluster;
    while (size > 1 && (int64_t(c.num_seqs) * size > 152 || c.vocab / 8 < size * kThr / 2)) size /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(c.num_seqs) * size);
    cfg.blockDim = dim3(kThr);
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
