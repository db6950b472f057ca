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
// leaves its result in the shared memory of every CTA of the cluster; behind one
// cluster barrier each warp joins all of them in the same order and takes the
// decisions itself.  Only rank 0 writes.  A second kernel joins the sequences'
// lists.
#include <cooperative_groups.h>

#include "pa_device.h"
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

// The largest logit and the sum of 2^((x - largest) c); with a NaN or an
// infinite largest one the sum is not finite.
struct Stat {
    float top, sum;
};
// What a warp found in a pass.
struct Slot {
    Stat p, q;
    float key;  // of the best candidate for the next token, or a sum
    int at;     // where the largest logit (greedy) or the best candidate is
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

template <int N> __device__ inline void take(Stat& s, const float (&x)[N], float c) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
    if (top > s.top) {
        s.sum *= ex2((s.top - top) * c);
        s.top = top;
    }
    if (s.top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < N; ++i) s.sum += ex2((x[i] - s.top) * c);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) s.sum += x[i] != x[i] ? x[i] : 0.f;
    }
}
// s over the warp's lanes.
__device__ inline Stat over_warp(Stat s, float c) {
    float top = s.top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // a lane that saw nothing, or only -infinity, adds what it has: 0, or a NaN
    s.sum = warp_sum(s.top > -INFINITY ? s.sum * ex2((s.top - top) * c) : s.sum);
    s.top = top;
    return s;
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
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        better(key, at, __shfl_xor_sync(0xffffffffu, key, o), __shfl_xor_sync(0xffffffffu, at, o));
}

template <typename T> __global__ void __launch_bounds__(kThr, 1) verify_walk(const VerifyCall a) {
    constexpr int kAhead = Elt<T>::kVec / 2;  // units of eight logits whose loads a thread has in flight
    __shared__ Slot inbox[2][kMaxCluster * kWarps];
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
    __syncthreads();

    int phase = 0;
    // Leaves the warp's result with every CTA of the cluster; `meanwhile` runs
    // before the others' have come.  Returns all of them, a slot to be read again
    // only before the next exchange but one.
    auto exchange = [&](const Slot& mine, auto&& meanwhile) -> const Slot* {
        if (lane < C) *cluster.map_shared_rank(&inbox[phase][rank * kWarps + warp], lane) = mine;
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        meanwhile();
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        const Slot* all = inbox[phase];
        phase ^= 1;
        return all;
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
        // the lane's child: its logits
        float x_mine = 0.f, y_mine = 0.f;
        auto look = [&] {
            if ((children >> lane) & 1u) {
                const int token = tokens[base + lane];
                x_mine = Elt<T>::f(row[token]);
                if (q_row) y_mine = Elt<T>::f(q_row[token]);
            }
        };
        look();
        const Span sp = span_of(row, V);
        const bool q_wide = q_row && wide_at(q_row + sp.head);
        Slot mine = {{-INFINITY, 0.f}, {-INFINITY, 0.f}, -INFINITY, V};
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
                        take<8>(mine.p, x, c);
                        if (greedy) {
                            const int at = sp.head + 8 * (i + k * workers);
#pragma unroll
                            for (int e = 0; e < 8; ++e) first_place(x[e], at + e);
                        }
                        if (q_row) {
                            v[k].get(x);
                            take<8>(mine.q, x, c);
                        }
                    }
            },
            [&](int at) {
                float x[1] = {Elt<T>::f(row[at])};
                take<1>(mine.p, x, c);
                if (greedy) first_place(x[0], at);
                if (q_row) {
                    x[0] = Elt<T>::f(q_row[at]);
                    take<1>(mine.q, x, c);
                }
            });
        mine.p = over_warp(mine.p, c);
        if (q_row) mine.q = over_warp(mine.q, c);
        if (greedy) better_over_warp(mine.key, mine.at);
        const Slot* all = exchange(mine, [&] {  // the row that the walk most likely goes on to
            if (!children) return;
            const int t = base + __ffs(children) - 1;
            prefetch(reinterpret_cast<const char*>(logits + int64_t(r0 + t) * a.logits_stride), int64_t(V) * sizeof(T));
            if (draft && t + 1 < rows && parents[t + 1] == t)
                prefetch(reinterpret_cast<const char*>(draft + int64_t(r0 + t) * a.draft_stride), int64_t(V) * sizeof(T));
        });
        Stat P = {-INFINITY, 0.f}, Q = {-INFINITY, 0.f};
        float top_key = -INFINITY;
        int top_at = V;
        for (int i = lane; i < C * kWarps; i += 32) {
            const Slot o = all[i];
            auto join = [&](Stat& x, const Stat& y) {
                const float top = fmaxf(x.top, y.top);
                x.sum = (x.top > -INFINITY ? x.sum * ex2((x.top - top) * c) : x.sum) +
                        (y.top > -INFINITY ? y.sum * ex2((y.top - top) * c) : y.sum);
                x.top = top;
            };
            join(P, o.p);
            if (q_row) join(Q, o.q);
            if (greedy) better(top_key, top_at, o.key, o.at);
        }
        P = over_warp(P, c);
        if (q_row) Q = over_warp(Q, c);
        if (greedy) better_over_warp(top_key, top_at);
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
                if (p > 0.f && a.uniform[r0 + t] * q < p) went = t;
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
                sum = 0.f;
                for (int i = lane; i < C * kWarps; i += 32) sum += sums[i].key;
                sum = warp_sum(sum);
                if (sum > 0.f) {
                    used = more;
                    mass = sum;
                }
            }
        }
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
            const float q_s = used * q_of;
            float best = 0.f;
            int best_at = V;
            // p / e against the best one so far: a division only where a product says that it may be better
            auto weigh = [&](float p, float e, int at) {
                if (!(p > best * e * 0.999999f)) return;
                const float key = p / e;
                if (!(key > best || (key == best && at < best_at))) return;
                for (int k = 0; k < dropped; ++k)
                    if (removed[k] == at) return;
                best = key;
                best_at = at;
            };
            auto left = [&](float x, float y) {
                const float p = ex2((x - P.top) * c) * p_of;
                return q_s > 0.f ? fmaxf(p - ex2((y - Q.top) * c) * q_s, 0.f) : p;
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
#pragma unroll
                            for (int e = 0; e < 8; ++e) weigh(left(x8[e], q_s > 0.f ? y8[e] : 0.f), e8[e], at + e);
                        }
                },
                [&](int at) { weigh(left(Elt<T>::f(row[at]), q_s > 0.f ? Elt<T>::f(q_row[at]) : 0.f), noise[at], at); });
            better_over_warp(best, best_at);
            mine.key = best;
            mine.at = best_at;
            const Slot* picks = exchange(mine, [] {});
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
