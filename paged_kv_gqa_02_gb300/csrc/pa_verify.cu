// pa_verify.cu -- which drafted tokens the target's distribution accepts, and
// the token behind them.
//
// A cluster of CTAs walks one sequence's tree.  Only the rows that the walk
// visits are read: their logits' largest value and sum in one pass (the
// draft's row in the same one), then scalars alone decide about the children.
// After k rejections what is left of p is max(p - a q, 0) / M with
//   a_1 = 1, M_k = sum max(p - a_k q, 0), a_{k+1} = a_k + M_k,
// which is k times "subtract q, clamp, normalise" in one step, so a rejection
// costs one sum over the vocabulary whatever came before it, and certain drafts
// (q a single token) cost none.  The next token is the largest p_i / e_i for
// exponential e_i: a comparison of single terms, which rounding can turn only
// where two are within a few units of 2^-24 of each other, while a search in
// running sums would meet a border every few 2^-24 in a vocabulary's tail.
//
// All CTAs of a cluster take each decision themselves, from sums that each
// gathers from all in the same order; only rank 0 writes.  A second kernel
// joins the sequences' lists.
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
constexpr int kMaxCluster = 8;
constexpr int kMaxDrafts = 1024;  // rows of a sequence
constexpr int kAhead = 2;         // units of eight logits whose loads a thread has in flight
constexpr int kPackThr = 1024;
constexpr float kBiggest = 3.402823466e38f;

// What a pass over a row leaves: the largest logit and its first place, the sum
// of 2^((x - largest) c), and whether every value was below infinity and none NaN.
struct Stat {
    float top, sum;
    int at, fine;
};

// A candidate for the next token.
struct Pick {
    float key;
    int at;
};

struct Slot {  // what a CTA shows the others after a pass
    Stat target, draft;
    Pick pick;
    float mass;
};

// A row of the vocabulary as each thread reads it: single elements up to the
// first 16-byte boundary, units of eight, single elements.
struct Span {
    int head, units, vocab;
};
template <typename T> __device__ inline Span span_of(const T* row, int vocab) {
    Span s;
    const int off = int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    s.head = min(vocab, off ? int(16 / sizeof(T)) - off : 0);
    s.units = (vocab - s.head) / 8;
    s.vocab = vocab;
    return s;
}

template <typename T> struct Unit {
    uint4 v[8 / Elt<T>::kVec];
};
// Eight elements from p: 16-byte loads where p is aligned.
template <typename T> __device__ inline void load8(const T* p, bool wide, float (&x)[8]) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < 8 / Elt<T>::kVec; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
            vec_to_f32<T>(v, x + i * Elt<T>::kVec);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = Elt<T>::f(p[i]);
    }
}
template <typename T> __device__ inline bool wide_at(const T* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

__device__ inline void take(Stat& s, const float* x, int n, int at, float c) {
    float top = x[0];
    for (int i = 1; i < n; ++i) top = fmaxf(top, x[i]);
    if (top > s.top) {
        s.sum *= ex2((s.top - top) * c);
        s.top = top;
        for (int i = n - 1; i >= 0; --i)
            if (x[i] == top) s.at = at + i;
    }
    for (int i = 0; i < n; ++i) {
        s.fine &= x[i] <= kBiggest;
        if (x[i] > -INFINITY) s.sum += ex2((x[i] - s.top) * c);
    }
}

__device__ inline Stat join(const Stat& a, const Stat& b, float c) {
    Stat r;
    const bool second = b.top > a.top || (b.top == a.top && b.at < a.at);
    r.top = second ? b.top : a.top;
    r.at = second ? b.at : a.at;
    r.fine = a.fine & b.fine;
    r.sum = 0.f;
    if (a.top > -INFINITY) r.sum += a.sum * ex2((a.top - r.top) * c);
    if (b.top > -INFINITY) r.sum += b.sum * ex2((b.top - r.top) * c);
    return r;
}
__device__ inline Pick join(const Pick& a, const Pick& b) {
    return b.key > a.key || (b.key == a.key && b.at < a.at) ? b : a;
}
__device__ inline Stat shuffled(const Stat& s, int o) {
    return Stat{__shfl_xor_sync(0xffffffffu, s.top, o), __shfl_xor_sync(0xffffffffu, s.sum, o),
                __shfl_xor_sync(0xffffffffu, s.at, o), __shfl_xor_sync(0xffffffffu, s.fine, o)};
}
__device__ inline Pick shuffled(const Pick& s, int o) {
    return Pick{__shfl_xor_sync(0xffffffffu, s.key, o), __shfl_xor_sync(0xffffffffu, s.at, o)};
}

template <typename T> __global__ void __launch_bounds__(kThr) verify_walk(const VerifyCall a) {
    __shared__ Slot warp_slots[kWarps];
    __shared__ Slot slots[2];
    __shared__ int removed[kMaxDrafts];
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
    const int V = a.vocab;
    const int32_t* tokens = a.tokens + r0;
    const int32_t* parents = a.parents + r0;
    if (rank == 0)
        for (int t = 1 + tid; t < rows; t += kThr)
            if (parents[t] < 0 || parents[t] >= t || tokens[t] < 0 || tokens[t] >= V)
                flag(a.dev_status, PA_DEV_BAD_INDEX);
    const float heat = a.temperature[s];
    const bool greedy = !(heat > 0.f);
    const float c = greedy ? kLog2e : fminf(kLog2e / heat, kBiggest);
    const T* const logits = static_cast<const T*>(a.logits);
    const T* const draft = greedy ? nullptr : static_cast<const T*>(a.draft);
    int phase = 0;

    // the first child of `here` behind row t with a token of the vocabulary, or `rows`
    auto child_after = [&](int here, int t) {
        for (int base = t + 1; base < rows; base += 32) {
            const int r = base + lane;
            const unsigned m =
                __ballot_sync(0xffffffffu, r < rows && parents[r] == here && tokens[r] >= 0 && tokens[r] < V);
            if (m) return base + __ffs(m) - 1;
        }
        return rows;
    };
    // what all threads of the cluster found: one slot each, joined in a fixed order
    auto gather = [&](Slot mine, auto&& joined) {
        if (lane == 0) warp_slots[warp] = mine;
        __syncthreads();
        if (tid == 0) {
            Slot all = warp_slots[0];
            for (int w = 1; w < kWarps; ++w) joined(all, warp_slots[w]);
            slots[phase] = all;
        }
        cluster.sync();
        Slot all = *cluster.map_shared_rank(&slots[phase], 0);
        for (int r = 1; r < C; ++r) joined(all, *cluster.map_shared_rank(&slots[phase], r));
        phase ^= 1;  // a slot is written again only behind the next pass's barrier
        return all;
    };
    // f(first index, eight or one) over the row's units, the cluster's threads in turn
    auto over = [&](const Span& sp, auto&& f) {
#pragma unroll kAhead
        for (int i = rank * kThr + tid; i < sp.units; i += C * kThr) f(sp.head + 8 * i, 8);
        const int behind = sp.head + 8 * sp.units, single = sp.head + (V - behind);
        if (rank == C - 1 && tid < single) f(tid < sp.head ? tid : behind + tid - sp.head, 1);
    };

    int here = 0, count = 0, next = -1;
    for (;;) {
        if (rank == 0 && tid == 0) a.accepted[r0 + count] = r0 + here;
        ++count;
        const T* const row = logits + int64_t(r0 + here) * a.logits_stride;
        int t = child_after(here, here);
        const T* const q_row = draft && t < rows ? draft + int64_t(r0 + here) * a.draft_stride : nullptr;
        const Span sp = span_of(row, V);
        const bool q_wide = q_row && wide_at(q_row + sp.head);
        Slot mine = {};
        mine.target = mine.draft = Stat{-INFINITY, 0.f, V, 1};
        over(sp, [&](int at, int n) {
            float x[8], y[8];
            if (n == 8) {
                load8(row + at, true, x);
                if (q_row) load8(q_row + at, q_wide, y);
                take(mine.target, x, 8, at, c);
                if (q_row) take(mine.draft, y, 8, at, c);
            } else {
                x[0] = Elt<T>::f(row[at]);
                take(mine.target, x, 1, at, c);
                if (q_row) {
                    y[0] = Elt<T>::f(q_row[at]);
                    take(mine.draft, y, 1, at, c);
                }
            }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            mine.target = join(mine.target, shuffled(mine.target, o), c);
            if (q_row) mine.draft = join(mine.draft, shuffled(mine.draft, o), c);
        }
        const Slot all = gather(mine, [&](Slot& x, const Slot& y) {
            x.target = join(x.target, y.target, c);
            x.draft = join(x.draft, y.draft, c);
        });
        const Stat P = all.target, Q = all.draft;
        if (!P.fine || !(P.top > -INFINITY) || (q_row && (!Q.fine || !(Q.top > -INFINITY)))) {
            if (rank == 0 && tid == 0) flag(a.dev_status, PA_DEV_BAD_VALUE);
            break;
        }
        // what is left of p is max(p - used q, 0) / mass
        double used = 0, mass = 1;
        int dropped = 0;  // certain drafts rejected here
        const double c64 = c;
        const float p_of = 1.f / P.sum, q_of = q_row ? 1.f / Q.sum : 0.f;
        bool went = false;
        while (t < rows) {
            const int token = tokens[t];
            if (greedy) {
                went = token == P.at;
            } else {
                const double x = Elt<T>::f(row[token]);
                double p = exp2((x - P.top) * c64) / P.sum, q = 1;
                bool again = false;
                if (q_row) {
                    q = exp2((double(Elt<T>::f(q_row[token])) - Q.top) * c64) / Q.sum;
                    p = fmax(p - used * q, 0.0) / mass;
                } else {
                    for (int i = lane; i < dropped; i += 32) again |= removed[i] == token;
                    again = __any_sync(0xffffffffu, again);
                    p = again ? 0 : p / mass;
                }
                went = p > 0 && double(a.uniform[r0 + t]) * q < p;
                if (!went && q_row) {
                    const double more = used + mass;
                    const float p_s = p_of, q_s = float(more * q_of);
                    float sum = 0.f;
                    over(sp, [&](int at, int n) {
                        float x8[8], y8[8];
                        if (n == 8) {
                            load8(row + at, true, x8);
                            load8(q_row + at, q_wide, y8);
                        } else {
                            x8[0] = Elt<T>::f(row[at]);
                            y8[0] = Elt<T>::f(q_row[at]);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i < n)
                                sum += fmaxf(ex2((x8[i] - P.top) * c) * p_s - ex2((y8[i] - Q.top) * c) * q_s, 0.f);
                    });
                    Slot m = {};
                    m.mass = warp_sum(sum);
                    const Slot sums = gather(m, [](Slot& x, const Slot& y) { x.mass += y.mass; });
                    if (sums.mass > 0.f) {
                        used = more;
                        mass = sums.mass;
                    }
                } else if (!went && !again && mass - p * mass > 0) {
                    mass -= p * mass;
                    __syncthreads();  // all warps have looked through the list
                    if (tid == 0) removed[dropped] = token;
                    ++dropped;
                    __syncthreads();
                }
            }
            if (went) break;
            t = child_after(here, t);
        }
        if (went) {
            here = t;
            continue;
        }
        if (greedy) {
            next = P.at;
            break;
        }
        const float* const noise = a.noise + int64_t(s) * V;
        const bool e_wide = wide_at(noise + sp.head);
        const float q_s = used > 0 ? float(used * q_of) : 0.f;
        Pick best = {0.f, V};
        over(sp, [&](int at, int n) {
            float x[8], y[8], e[8];
            if (n == 8) {
                load8(row + at, true, x);
                if (q_s > 0.f) load8(q_row + at, q_wide, y);
                load8(noise + at, e_wide, e);
            } else {
                x[0] = Elt<T>::f(row[at]);
                if (q_s > 0.f) y[0] = Elt<T>::f(q_row[at]);
                e[0] = noise[at];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= n) continue;
                float p = ex2((x[i] - P.top) * c) * p_of;
                if (q_s > 0.f) p = fmaxf(p - ex2((y[i] - Q.top) * c) * q_s, 0.f);
                const float key = p / e[i];
                if (key > best.key || (key == best.key && p > 0.f && at + i < best.at)) {
                    bool out = false;
                    for (int k = 0; k < dropped; ++k) out |= removed[k] == at + i;
                    if (!out) best = Pick{key, at + i};
                }
            }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = join(best, shuffled(best, o));
        Slot m = {};
        m.pick = best;
        const Slot picked = gather(m, [](Slot& x, const Slot& y) { x.pick = join(x.pick, y.pick); });
        if (picked.pick.key > 0.f)
            next = picked.pick.at;
        else if (rank == 0 && tid == 0)
            flag(a.dev_status, PA_DEV_BAD_VALUE);
        break;
    }
    if (rank == 0 && tid == 0) {
        a.accepted_cu[s + 1] = count;
        a.next_tokens[s] = next;
    }
    cluster.sync();  // nobody leaves while another may read its slots
}

// Joins the sequences' lists: the walk left counts in accepted_cu and each
// list at its sequence's own rows, which lie at or behind its place in the
// joined one, so a tile of places can be read, then written, in ascending order.
__global__ void __launch_bounds__(kPackThr) verify_pack(const VerifyCall a) {
    __shared__ int sums[kPackThr / 32];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int base = 0;
    if (tid == 0) a.accepted_cu[0] = 0;
    for (int s0 = 0; s0 < a.num_seqs; s0 += kPackThr) {
        const int s = s0 + tid;
        const int n = s < a.num_seqs ? a.accepted_cu[s + 1] : 0;
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
        for (int w = 0; w < kPackThr / 32; ++w) {
            if (w < warp) v += sums[w];
            all += sums[w];
        }
        if (s < a.num_seqs) {
            a.accepted_cu[s + 1] = base + v;
            if (a.new_lens) a.new_lens[s] = a.context_lens[s] + n;
        }
        base += all;
    }
    __syncthreads();
    const int total = min(base, a.total_rows);
    for (int j0 = 0; j0 < total; j0 += kPackThr) {
        const int j = j0 + tid;
        int row = -1;
        if (j < total) {
            int lo = 0, hi = a.num_seqs - 1;  // the sequence: the last that begins at or before j and is not empty
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (a.accepted_cu[mid + 1] > j)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            row = a.accepted[a.cu_lens[lo] + j - a.accepted_cu[lo]];
        }
        __syncthreads();
        if (j < total) a.accepted[j] = row;
        __syncthreads();
    }
    for (int j = total + tid; j < a.total_rows; j += kPackThr) a.accepted[j] = -1;
}

template <typename T> cudaError_t launch_walk(const VerifyCall& c, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    int size = kMaxCluster;
    while (size > 1 && int64_t(c.num_seqs) * size > 2 * 152) size /= 2;
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
