// moe_gate.cu -- the choice of experts from the router's logits and its gradient, and the (token,
// choice) pairs sorted by expert (include/swiglu_tokens.h).
//
// One GB300, device times: the choice of 8 of 128 experts for 65536 tokens (fp32, 38 MB) 12.8 us (bf16 11.3;
// 64 experts 8.7, 8.5).  Nothing is saturated: 147 instructions a token keep the integer pipe 66 % and the issue
// slots 50 % busy, with 41 % of an SM's warps (64 registers) and HBM at 26 %; each round waits for the one
// before.  Its gradient 7.1 us, and 12 where it needs all experts' probabilities (75 MB), both near HBM's rate;
// 40961 tokens of 61 experts, bf16, 5.8 us for 2.0 of traffic, 2-byte accesses.  The sort of 16384 pairs 4.7 us, of
// 131072 9.1, of 1048576 43 to 55 (64 and 682 experts).
#include <cooperative_groups.h>

#include <algorithm>

#include "rows.cuh"
#include "swiglu_tokens.h"

namespace swiglu {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxExperts = 1024;
constexpr int kGateThreads = 128;

struct Gate {
    const void* logits;
    void* dlogits;
    int* ids;
    float* gates;
    const float* dgates;
    int64_t ld, lddl, T;
    int E, k, renorm;
};

// Order-preserving key of a logit: larger logit, larger key; NaN lowest but above 0, which is an
// expert that is switched off.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (isnan(v)) return 1;
    if (v == -INFINITY) return 0;
    const uint32_t u = __float_as_uint(v + 0.f);           // -0 counts as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// A token's logits belong to a group of G lanes of a warp.  A lane has OWN of them, in runs of RUN
// consecutive experts; its i-th one (rising with i):
template <int G, int RUN>
__device__ __forceinline__ int expert(int i) {
    return (i / RUN * G + (threadIdx.x & (G - 1))) * RUN + i % RUN;
}
template <int G>
struct Group {
    static __device__ __forceinline__ int lane() { return threadIdx.x & (G - 1); }
    static __device__ __forceinline__ int64_t token() { return ((int64_t)blockIdx.x * kGateThreads + threadIdx.x) / G; }
    static __device__ __forceinline__ uint32_t max(uint32_t v) {
        if constexpr (G == 32) {
            v = __reduce_max_sync(0xffffffffu, v);
        } else {
#pragma unroll
            for (int o = G / 2; o; o >>= 1) v = ::max(v, __shfl_xor_sync(0xffffffffu, v, o));
        }
        return v;
    }
    static __device__ __forceinline__ float max(float v) {
#pragma unroll
        for (int o = G / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
    static __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    template <class V>
    static __device__ __forceinline__ V of(V v, int lane) { return __shfl_sync(0xffffffffu, v, lane, G); }
};

template <class T, int N>
struct alignas(N * sizeof(T)) Run {
    T v[N];
};

// The lane's own logits; minus infinity past the row's end (and for a token past the last).  A run is one
// load (the gradient of 65536 tokens of 128 experts, fp32: 12.3 us with runs of 4, 13.7 without).
template <class T, int OWN, int G, int RUN>
__device__ __forceinline__ void load_logits(float* v, const Gate& a, int64_t t) {
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const int E = t < a.T ? a.E : 0;
#pragma unroll
    for (int i = 0; i < OWN; i += RUN) {
        const int e = expert<G, RUN>(i);
        Run<T, RUN> r;
        if (e < E) r = *reinterpret_cast<const Run<T, RUN>*>(row + e);
#pragma unroll
        for (int j = 0; j < RUN; ++j) v[i + j] = e < E ? to_f32(r.v[j]) : -INFINITY;
    }
}

template <int OWN, int G>
__device__ __forceinline__ float exp_sum(const float* v, float top) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < OWN; ++i) sum += expf(v[i] - top);
    return Group<G>::sum(sum);
}

// Batcher's odd-even merge sort, largest first.  Every index is a template's, so that the words stay
// in registers.
template <int A, int B>
__device__ __forceinline__ void order(uint32_t* w) {
    const uint32_t hi = max(w[A], w[B]), lo = min(w[A], w[B]);
    w[A] = hi, w[B] = lo;
}
template <int I, int END, int R>
__device__ __forceinline__ void order_pairs(uint32_t* w) {
    if constexpr (I + R < END) {
        order<I, I + R>(w);
        order_pairs<I + 2 * R, END, R>(w);
    }
}
// Merges the halves of w[AT] .. w[AT + N - 1], of which every R-th word is meant.
template <int AT, int N, int R>
__device__ __forceinline__ void merge_words(uint32_t* w) {
    if constexpr (2 * R < N) {
        merge_words<AT, N, 2 * R>(w);
        merge_words<AT + R, N, 2 * R>(w);
        order_pairs<AT + R, AT + N, R>(w);
    } else {
        order<AT, AT + R>(w);
    }
}
template <int AT, int N>
__device__ __forceinline__ void sort_words(uint32_t* w) {
    if constexpr (N > 1) {
        sort_words<AT, N / 2>(w);
        sort_words<AT + N / 2, N / 2>(w);
        merge_words<AT, N, 1>(w);
    }
}

// The choices by whole keys, one after the other: the largest that is left, of equal ones the lowest
// index.  Lane j has the choice j0 + j of each run of G; the gates of a run that is not the last wait
// in memory, as exponentials, until all are known.
template <class T, int OWN, int G>
__device__ __noinline__ void choose_by_keys(const Gate& a, int64_t t) {
    const int lane = Group<G>::lane();
    float v[OWN], top = -INFINITY;
    uint32_t key[OWN];
    load_logits<T, OWN, G, 1>(v, a, t);
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        top = fmaxf(top, v[i]);
        key[i] = expert<G, 1>(i) < a.E ? logit_key(v[i]) : 0;
    }
    top = Group<G>::max(top);
    if (top == -INFINITY) top = 0.f;
    const float total = exp_sum<OWN, G>(v, top);
    int* ids = a.ids + t * a.k;
    float* gates = a.gates + t * a.k;
    float chosen = 0.f, p;
    int mine;
    for (int j0 = 0; j0 < a.k; j0 += G) {
        const int n = min(G, a.k - j0);
        mine = -1, p = 0.f;
        for (int j = 0; j < n; ++j) {
            uint32_t best = key[0];
            float value = v[0];
            int at = expert<G, 1>(0);
#pragma unroll
            for (int i = 1; i < OWN; ++i)
                if (key[i] > best) best = key[i], value = v[i], at = expert<G, 1>(i);
            const uint32_t high = Group<G>::max(best);
            const int e = kMaxExperts - (int)Group<G>::max(best == high ? (uint32_t)(kMaxExperts - at) : 0u);
            value = Group<G>::of(value, e & (G - 1));
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                if (e == expert<G, 1>(i)) key[i] = 0;
            if (lane == j && high != 0) mine = e, p = value;
        }
        p = mine < 0 ? 0.f : expf(p - top);
        chosen += Group<G>::sum(p);
        if (t < a.T && lane < n) {
            ids[j0 + lane] = mine;
            if (j0 + G < a.k) gates[j0 + lane] = mine < 0 ? -1.f : p;
        }
    }
    const float by = a.renorm ? chosen + 0.f * total : total;          // total: NaN where a logit is
    if (t >= a.T) return;
    const int last = (a.k - 1) / G * G + lane;
    if (last < a.k) gates[last] = mine < 0 ? 0.f : p / by;
    for (int j = last - G; j >= 0; j -= G) gates[j] = gates[j] < 0.f ? 0.f : gates[j] / by;
}

// top_k of more than 32 (4096 tokens, 40 of 512 experts: 34 us for 1.5 of traffic, a maximum over the warp and a pass over the
// lane's keys for each choice).
template <class T, int OWN>
__global__ void __launch_bounds__(kGateThreads) moe_gate_fwd_keys_kernel(const __grid_constant__ Gate a) {
    after_previous();
    choose_by_keys<T, OWN, 32>(a, Group<32>::token());
}

// Order-preserving key of a logit that is no NaN; 0 and -0 have one.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// A lane's words without the first, where the group's largest is hers.
template <int KEEP>
__device__ __forceinline__ void pop(uint32_t* word, uint32_t high) {
    if (word[0] != high) return;
#pragma unroll
    for (int i = 0; i + 1 < KEEP; ++i) word[i] = word[i + 1];
    word[KEEP - 1] = 0;
}

// The choices by words, where some are alike in them but not in their logits: among the chosen
// (their order), or beyond the last one (border: `next`, and who is chosen).  Puts both right; false where
// too many beyond the last are alike in their words but differ, or a lane's KEEP words do not show them.
template <int OWN, int G, int KEEP>
__device__ __forceinline__ bool settle(const Gate& a, int64_t t, uint32_t* word, uint32_t next, bool border, uint32_t mine, int& e, float& value) {
    constexpr uint32_t kAll = OWN * G, kIndex = 2 * kAll - 1;
    const int lane = Group<G>::lane();
    const float* row = static_cast<const float*>(a.logits) + t * a.ld;
    const uint32_t last = Group<G>::of(mine, a.k - 1);
    const bool alike = lane < a.k && (mine ^ last) <= kIndex;
    uint32_t key = order_key(value);
    // the ones beyond, one by one: in the place of the last of those chosen that are alike, if larger.  They come
    // by falling word, so of equal logits by rising index, until a lane has no words left: what it would show
    // next is not known.
    uint32_t least = 0;
    bool more = border, ran_out = false;
    for (int turn = 0; turn < 4; ++turn) {
        if (!__any_sync(0xffffffffu, more)) break;
        const int e2 = (int)(kAll - (next & kIndex));
        const float v2 = more ? row[e2] : -INFINITY;
        least = ~Group<G>::max(alike ? ~key : 0u);
        const int worst = (int)Group<G>::max(alike && key == least ? (uint32_t)e + 1 : 0u) - 1;
        if (more && alike && e == worst && order_key(v2) > least) e = e2, value = v2, key = order_key(v2);
        if (more) pop<KEEP>(word, next);
        next = Group<G>::max(word[0]);
        if constexpr (KEEP < OWN) ran_out = Group<G>::max(word[0] == 0 ? 1u : 0u) != 0;
        more = more && !ran_out && (next ^ last) <= kIndex;
    }
    border = more || ran_out;
    bool settled = true;
    if (__any_sync(0xffffffffu, border)) {                 // the rest: whether any is larger than the least chosen (equal ones come after it)
        float v[OWN], larger = 0.f;
        load_logits<float, OWN, G, 1>(v, a, t);
        least = ~Group<G>::max(alike ? ~key : 0u);
#pragma unroll
        for (int i = 0; i < OWN; ++i) larger += expert<G, 1>(i) < a.E && order_key(v[i]) > least;
        larger = Group<G>::sum(larger - (float)(lane < a.k && key > least));
        settled = !border || larger == 0.f;
    }
    int rank = 0;
    for (int i = 0; i < a.k; ++i) {
        const uint32_t k2 = Group<G>::of(key, i);
        const int e2 = Group<G>::of(e, i);
        rank += k2 > key || (k2 == key && e2 < e);
    }
    const int e0 = e;
    const float v0 = value;
    for (int i = 0; i < a.k; ++i) {
        const int to = Group<G>::of(rank, i), e2 = Group<G>::of(e0, i);
        const float v2 = Group<G>::of(v0, i);
        if (lane == to && lane < a.k) e = e2, value = v2;
    }
    return settled;
}

// top_k up to G.  An expert's word has its index in the lowest bits (from all experts down, so that of equal
// logits the lowest index is the largest word) and as many of the first bits of its key as there is room
// for: one maximum over the group finds the next choice and who has it, and a lane that keeps its words
// sorted shows only the first.  These are at least 21 bits, which is all of a 16-bit logit's key.  For fp32
// the order by words can be wrong only among keys alike in them, which `settle` puts right (24 bits for 128
// experts: one token in 600 of normal logits, for which choosing anew by whole keys held up the last warps: 15.3
// us instead of 12.6); where it cannot, or a logit is NaN, the warp chooses by whole keys.
template <class T, int OWN, int G>
__global__ void __launch_bounds__(kGateThreads, OWN > 16 ? 3 : 8) moe_gate_fwd_kernel(const __grid_constant__ Gate a) {
    after_previous();
    constexpr uint32_t kAll = OWN * G, kIndex = 2 * kAll - 1;
    constexpr int kKeep = OWN > G ? G + 1 : OWN;           // of a lane's words: the choice shows top_k + 1 at most
    const int64_t t = Group<G>::token();
    const int lane = Group<G>::lane();
    uint32_t word[OWN];
    float total = 0.f;
    {
        float v[OWN];
        load_logits<T, OWN, G, 1>(v, a, t);
        // Places past the row's end, minus infinity too, come after all the row's.  The sum makes each NaN
        // 0x7fffffff, whose key is the largest.
#pragma unroll
        for (int i = 0; i < OWN; ++i) word[i] = (order_key(v[i]) & ~kIndex) | (kAll - expert<G, 1>(i));
        if (!a.renorm) {
            float top = v[0];
#pragma unroll
            for (int i = 1; i < OWN; ++i) top = fmaxf(top, v[i]);
            top = Group<G>::max(top);
            total = exp_sum<OWN, G>(v, top == -INFINITY ? 0.f : top);
        }
    }
    sort_words<0, OWN>(word);
    bool again = word[0] > (0xffffffffu & ~kIndex);        // a NaN
    uint32_t mine = 0;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t high = Group<G>::max(word[0]);
        if (lane == j) mine = high;
        pop<kKeep>(word, high);
    }
    int e = lane < a.k ? (int)(kAll - (mine & kIndex)) : -1;
    float value = e < 0 || t >= a.T ? -INFINITY : to_f32(static_cast<const T*>(a.logits)[t * a.ld + e]);
    if constexpr (sizeof(T) == 4) {
        const uint32_t next = Group<G>::max(word[0]), after = Group<G>::of(mine, lane + 1);
        const float other = Group<G>::of(value, lane + 1);
        const bool inner = lane < a.k - 1 && (mine ^ after) <= kIndex && value != other;
        const bool border = Group<G>::of((mine ^ next) <= kIndex && value != -INFINITY, a.k - 1);
        if (__any_sync(0xffffffffu, inner || border)) again |= !settle<OWN, G, kKeep>(a, t, word, next, border, mine, e, value);
    }
    if (__any_sync(0xffffffffu, again)) return choose_by_keys<T, OWN, G>(a, t);
    const float top = Group<G>::of(value, 0);
    if (value == -INFINITY) e = -1;                        // off
    const float p = e < 0 ? 0.f : expf(value - top);
    if (a.renorm) total = Group<G>::sum(p);
    if (t < a.T && lane < a.k) {
        a.ids[t * a.k + lane] = e;
        a.gates[t * a.k + lane] = e < 0 ? 0.f : p / total;
    }
}

// dlogits_e = q_j (g_j - s) where e is choice j; else 0 (renormalize) or -p_e s.  First the latter for
// every expert, then the choices in their places, which need no search for who has which (with a compare
// for every choice and expert, and match.any for repeated ones, 65536 tokens of 128 experts took 20 us
// instead of 7.3).
template <class T, int OWN, int G, int RUN>
__global__ void __launch_bounds__(kGateThreads) moe_gate_bwd_kernel(const __grid_constant__ Gate a) {
    after_previous();
    __shared__ uint8_t owners[kGateThreads / G][OWN * G];
    const int lane = Group<G>::lane();
    // q and g of choice j0 + lane of token t; its id, -1 where it is no expert
    struct Choice {
        int id;
        float q, g;
    };
    auto load = [&](int64_t t, int j0) {
        Choice c{-1, 0.f, 0.f};
        if (t < a.T && j0 + lane < a.k) {
            const int64_t at = t * a.k + j0 + lane;
            c = Choice{a.ids[at], a.gates[at], a.dgates[at]};
            if ((unsigned)c.id >= (unsigned)a.E) c = Choice{-1, 0.f, 0.f};
        }
        return c;
    };
    const int64_t t = Group<G>::token();
    float d[OWN], s = 0.f;
    if (!a.renorm) load_logits<T, OWN, G, RUN>(d, a, t);
    Choice c = load(t, 0);
    // an index twice (or choices that one load does not hold) makes each expert add up its own
    uint8_t* owner = owners[threadIdx.x / G];
    if (c.id >= 0) owner[c.id] = (uint8_t)lane;
    __syncwarp();
    const bool sums = __any_sync(0xffffffffu, c.id >= 0 && owner[c.id] != lane) || a.k > G;
    s = c.q * c.g;
    for (int j0 = G; j0 < a.k; j0 += G) {
        const Choice more = load(t, j0);
        s += more.q * more.g;
    }
    s = Group<G>::sum(s);
    if (a.renorm) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) d[i] = 0.f;
    } else {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < OWN; ++i) top = fmaxf(top, d[i]);
        top = Group<G>::max(top);
        if (top == -INFINITY) top = 0.f;
#pragma unroll
        for (int i = 0; i < OWN; ++i) sum += d[i] = expf(d[i] - top);
        sum = Group<G>::sum(sum);
        const float by = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < OWN; ++i) d[i] *= by;          // p
    }
    const float place = c.q * (c.g - s);
    if (sums) {
        float up[OWN];
#pragma unroll
        for (int i = 0; i < OWN; ++i) up[i] = 0.f;
        for (int j0 = 0; j0 < a.k; j0 += G) {
            if (j0 > 0) c = load(t, j0);
            const float u = a.renorm ? c.q * (c.g - s) : c.g;
            for (int j = 0; j < min(G, a.k - j0); ++j) {
                const int e = Group<G>::of(c.id, j);
                const float w = Group<G>::of(u, j);
#pragma unroll
                for (int i = 0; i < OWN; ++i)
                    if (e == expert<G, RUN>(i)) up[i] += w;
            }
        }
#pragma unroll
        for (int i = 0; i < OWN; ++i) d[i] = a.renorm ? up[i] : d[i] * (up[i] - s);
        c.id = -1;
    } else if (!a.renorm) {
#pragma unroll
        for (int i = 0; i < OWN; ++i) d[i] *= -s;
    }
    T* out = static_cast<T*>(a.dlogits) + t * a.lddl;
#pragma unroll
    for (int i = 0; i < OWN; i += RUN) {
        Run<T, RUN> r;
#pragma unroll
        for (int j = 0; j < RUN; ++j) r.v[j] = from_f32<T>(d[i + j]);
        if (t < a.T && expert<G, RUN>(i) < a.E) *reinterpret_cast<Run<T, RUN>*>(out + expert<G, RUN>(i)) = r;
    }
    __syncwarp();
    if (c.id >= 0) out[c.id] = from_f32<T>(place);
}

// ---------------------------------------------------------------- sort

constexpr int kSortCtas = 8;
constexpr int kSortWarps = 32;

struct Sort {
    const int* ids;
    int *counts, *pos;
    int64_t n, per_warp;
    int E;
};

// Of n counts `ld` apart, a multiple of 4: each becomes the sum of those before it; returns the sum of all.
// Four loads at a time (one by one, the latencies add up: 0.5 us for 32 warps).
__device__ __forceinline__ int sum_before(int* p, int ld, int n) {
    int sum = 0;
    for (int w = 0; w < n; w += 4) {
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = p[(w + i) * ld];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[(w + i) * ld] = sum, sum += v[i];
    }
    return sum;
}
__device__ __forceinline__ void add_to_all(int* p, int ld, int n, int add) {
    for (int w = 0; w < n; w += 4) {
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = p[(w + i) * ld];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[(w + i) * ld] = v[i] + add;
    }
}

// Counting sort of the pairs by one cluster, in one launch.  Each warp has a run of consecutive pairs, 32
// at a time, and a count for each expert; the counts of all warps, added up over the warps before it and
// over the experts before, are where its first pair of each expert goes.  The lanes that have one expert
// find each other by a bit each in a word of it, so that the order does not depend on timing (131072
// pairs 9.1 us; by a vote a bit 15.2, by match.any 30).  Latencies bound it: four barriers, two of them the
// cluster's.
__global__ void __launch_bounds__(kSortWarps * 32) moe_sort_kernel(const Sort a) {
    extern __shared__ int smem[];
    after_previous();
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* mine = smem;                      // [E] this CTA's pairs of each expert
    int* base = mine + a.E;                // [E] first row of this CTA's pairs
    int* chunk = base + a.E;               // [32] pairs of 32 experts
    int* hist = chunk + 32;                // [warps][E]
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    int* own = hist + warp * a.E;
    unsigned* lanes = reinterpret_cast<unsigned*>(hist + (warps + warp) * a.E);        // [E] the lanes that have an expert
    for (int e = lane; e < a.E; e += 32) own[e] = 0, lanes[e] = 0;
    __syncwarp();
    const int64_t begin = ((int64_t)rank * warps + warp) * a.per_warp;
    const int64_t end = min(begin + a.per_warp, a.n);
    auto load = [&](int64_t p) {
        const int e = p < end ? a.ids[p] : -1;
        return (unsigned)e < (unsigned)a.E ? e : a.E;
    };
#pragma unroll 4
    for (int64_t p = begin + lane; p < end; p += 32) {
        const int e = load(p);
        if (e < a.E) atomicAdd(own + e, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) mine[e] = sum_before(hist + e, a.E, warps);
    cluster.sync();
    // per expert: the pairs of the CTAs before this one, and of all; then of the experts before it
    for (int e0 = warp * 32; e0 < a.E; e0 += warps * 32) {
        const int e = e0 + lane;
        int before = 0, all = 0;
        if (e < a.E) {
            for (int r = 0; r < ctas; ++r) {
                const int* theirs = cluster.map_shared_rank(mine, r);
                const int v = theirs[e];
                if (r < rank) before += v;
                all += v;
            }
            if (rank == 0) a.counts[e] = all;
        }
        int sum = all;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (e < a.E) base[e] = before + sum - all;
        if (lane == 31) chunk[e0 / 32] = sum;
    }
    cluster.sync();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int sum = base[e];
        for (int c = 0; c < e / 32; ++c) sum += chunk[c];
        add_to_all(hist + e, a.E, warps, sum);
    }
    __syncthreads();
    int next = load(begin + lane);
    for (int64_t p = begin + lane; p - lane < end; p += 32) {
        const int e = next;
        next = load(p + 32);
        if (e < a.E) atomicOr(lanes + e, 1u << lane);
        __syncwarp();
        const unsigned same = e < a.E ? lanes[e] : 0;
        const int first = e < a.E ? own[e] : -1;
        __syncwarp();
        if (e < a.E && same >> lane == 1) own[e] = first + __popc(same), lanes[e] = 0;          // the last of them
        if (p < end) a.pos[p] = first + __popc(same & ((1u << lane) - 1));
        __syncwarp();
    }
}

// ---------------------------------------------------------------- host side

struct LaunchGate {
    const Gate& a;
    bool bwd, runs;            // runs: whether rows can be moved four elements at a time
    cudaStream_t s;
    template <class T, int OWN, int G>
    cudaError_t go() const {
        const unsigned grid = (unsigned)((a.T * G + kGateThreads - 1) / kGateThreads);
        if (bwd)
            return runs ? launch_early(moe_gate_bwd_kernel<T, OWN, G, OWN < 4 ? OWN : 4>, grid, kGateThreads, 0, s, a)
                        : launch_early(moe_gate_bwd_kernel<T, OWN, G, 1>, grid, kGateThreads, 0, s, a);
        if constexpr (G == 32)
            if (a.k > G) return launch_early(moe_gate_fwd_keys_kernel<T, OWN>, grid, kGateThreads, 0, s, a);
        return launch_early(moe_gate_fwd_kernel<T, OWN, G>, grid, kGateThreads, 0, s, a);
    }
    // Few lanes a token share out its fixed costs best (65536 tokens, 8 of 128 experts, fp32, in L2: 12.0 us with
    // 8 lanes, 22.1 with 32; of 64 experts 8.7 and 21.9): as many as there are choices, each with up to 16 experts.
    template <class T>
    cudaError_t run() const {
        if (a.k <= 8 && a.E <= 128) return a.E <= 16 ? go<T, 2, 8>() : a.E <= 32 ? go<T, 4, 8>() : a.E <= 64 ? go<T, 8, 8>() : go<T, 16, 8>();
        if (a.k <= 16 && a.E <= 256) return a.E <= 64 ? go<T, 4, 16>() : a.E <= 128 ? go<T, 8, 16>() : go<T, 16, 16>();
        return a.E <= 128 ? go<T, 4, 32>() : a.E <= 512 ? go<T, 16, 32>() : go<T, 32, 32>();
    }
};

// Whether rows of `ld` elements of `n` bytes from p on, E of them used, can be moved four at a time.
bool in_runs(const void* p, int64_t ld, int64_t E, int n) { return n > 0 && !misaligned(p, 4 * n) && ld % 4 == 0 && E % 4 == 0; }

swiglu_status gate_check(const Gate& a, int64_t E, int64_t k, int type) {
    if (a.T < 0 || E <= 0 || k <= 0 || k > E) return fail(SWIGLU_ERR_INVALID_ARG, "gate: a size is negative or zero, or top_k above E");
    if (a.T >= (int64_t(1) << 31) || E > kMaxExperts)
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "gate: T must stay below 2^31, E up to 1024");
    if (type_bytes(type) == 0) return fail(SWIGLU_ERR_INVALID_ARG, "gate: unknown type");
    return SWIGLU_OK;
}

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

swiglu_status swiglu_moe_gate_fwd(const void* logits, int64_t ld, int32_t* ids, float* gates, int64_t T, int64_t E,
                                  int64_t top_k, int renormalize, int type, void* stream) {
    const int n = type_bytes(type);
    const Gate a{logits, nullptr, ids, gates, nullptr, ld, 0, T, (int)E, (int)top_k, renormalize != 0};
    swiglu_status rc = gate_check(a, E, top_k, type);
    if (rc != SWIGLU_OK || T == 0) return rc;
    if (!logits || !ids || !gates) return fail(SWIGLU_ERR_INVALID_ARG, "gate: a required pointer is null");
    if (ld < E) return fail(SWIGLU_ERR_INVALID_ARG, "gate: a row stride is smaller than E");
    if (misaligned(logits, n) || misaligned(ids, 4) || misaligned(gates, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "gate: a pointer is not aligned to its element");
    int sms;
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_MOE_GATE, s, [&] { return with_type(type, LaunchGate{a, false, false, s}); });
}

swiglu_status swiglu_moe_gate_bwd(const void* logits, int64_t ld, const int32_t* ids, const float* gates,
                                  const float* dgates, void* dlogits, int64_t lddl, int64_t T, int64_t E,
                                  int64_t top_k, int renormalize, int type, void* stream) {
    const int n = type_bytes(type);
    const Gate a{logits, dlogits, const_cast<int32_t*>(ids), const_cast<float*>(gates), dgates, ld, lddl, T, (int)E,
                 (int)top_k, renormalize != 0};
    const bool runs = (renormalize || in_runs(logits, ld, E, n)) && in_runs(dlogits, lddl, E, n);
    swiglu_status rc = gate_check(a, E, top_k, type);
    if (rc != SWIGLU_OK || T == 0) return rc;
    if ((!logits && !renormalize) || !ids || !gates || !dgates || !dlogits)
        return fail(SWIGLU_ERR_INVALID_ARG, "gate: a required pointer is null");
    if ((!renormalize && ld < E) || lddl < E) return fail(SWIGLU_ERR_INVALID_ARG, "gate: a row stride is smaller than E");
    if (misaligned(logits, n) || misaligned(dlogits, n) || misaligned(ids, 4) || misaligned(gates, 4) || misaligned(dgates, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "gate: a pointer is not aligned to its element");
    if (!renormalize && astride(logits, ld, dlogits, lddl, T))
        return fail(SWIGLU_ERR_INVALID_ARG, "gate: dlogits is in the logits' place with another row stride");
    int sms;
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_MOE_GATE, s, [&] { return with_type(type, LaunchGate{a, true, runs, s}); });
}

swiglu_status swiglu_moe_sort(const int32_t* ids, int32_t* counts, int32_t* pos, int64_t pairs, int64_t E,
                              void* stream) {
    if (pairs < 0 || E <= 0) return fail(SWIGLU_ERR_INVALID_ARG, "sort: a size is negative or zero");
    if (pairs >= (int64_t(1) << 31) || E > kMaxExperts)
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "sort: pairs must stay below 2^31, E up to 1024");
    if (!counts || (pairs > 0 && (!ids || !pos))) return fail(SWIGLU_ERR_INVALID_ARG, "sort: a required pointer is null");
    if (misaligned(ids, 4) || misaligned(counts, 4) || misaligned(pos, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "sort: a pointer is not aligned to its element");
    int sms;
    swiglu_status rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    int ctas = 1;
    while (ctas < kSortCtas && pairs > (int64_t)ctas * kSortWarps * 32) ctas *= 2;
    const int64_t runs = std::max<int64_t>(1, (pairs + 31) / 32), per_cta = (runs + ctas - 1) / ctas;
    const int most = E <= 768 ? kSortWarps : 24;           // of 227 KB
    const int warps = (int)std::min<int64_t>((per_cta + 3) / 4 * 4, most);
    const int64_t per_warp = (per_cta + warps - 1) / warps * 32;
    const Sort a{ids, counts, pos, pairs, per_warp, (int)E};
    const size_t smem = ((size_t)(2 * warps + 2) * E + 32) * sizeof(int);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_MOE_SORT, s, [&] {
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(moe_sort_kernel), smem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(warps * 32);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        return cudaLaunchKernelEx(&cfg, moe_sort_kernel, a);
    });
}

}  // extern "C"
