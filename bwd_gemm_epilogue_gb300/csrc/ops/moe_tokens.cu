// moe_tokens.cu -- tokens to their experts' rows and back, with the gates, dropout and the residual
// stream, the gradients of both, and dropout alone (include/swiglu_tokens.h).
//
// All of them move rows and compute little, so HBM bounds them where rows are whole 16-byte packs; one
// GB300, copies at 6.7 TB/s, device times without the launch's latency, which runs beside the kernel
// before (launch_early):
//   dispatch   8192 tokens to 2 of 8 experts, 4096 bf16 columns      30 us, 6.7 TB/s (with the sort 35)
//   combine    4096 tokens of 6 experts, 2048 bf16, dropout          24.8 us, 5.4 TB/s
//              8192 tokens of 2, 4096 bf16                           41.5 us, 6.5 TB/s
//   gradient   8192 tokens of 2, 4096 bf16, dropout                  49.6 us, 6.8 TB/s
//   dropout    11136 x 3584 bf16 into the residual stream            34.9 us, 6.9 TB/s
// A thread has a pack of the output, and what hides the latency of the rows, whose places have to be read
// first, is as many threads as an SM holds: two rows in flight a thread at 32 registers (combine above,
// 4 in flight at 40 and 48 registers: 28 and 27 us).  Rows off 16-byte boundaries start at another place
// of a pack each: those are put together from aligned pieces, about 20 instructions for 16 bytes, and
// these bound them (7 choices of 1021 columns, a tenth of them absent, 4099 tokens: combine bf16 with
// dropout 22.5 us for 10.4 of traffic, its gradient fp16 24.5 to 26.4 from GPU to GPU for 17.1; 2 of 4095 columns,
// 8192 tokens: combine 64 for 40.2, its gradient 68 for 50.2); fp32 rows, which are moved a column a thread
// instead: the dispatch's gradient 24.9 for 20.8, the combine's 39 for 34.1.
#include <algorithm>
#include <type_traits>

#include "dropout.cuh"
#include "swiglu_tokens.h"

namespace swiglu {
namespace {

constexpr int kMaxTop = 1024;
constexpr int kThreads = 256;

// How the rows of a call lie: all on 16-byte boundaries; off them, but each row alike in all tensors (of
// one row a token only: dropout); off them; or off them, fp32, and moved in singles, which takes fewer
// instructions than shifted packs but would compute a dropout's bits four times over.
enum Lie { kWhole, kAlike, kShifted, kApart };

// ---------------------------------------------------------------- rows to tokens

struct Gather {
    const void *rows, *add;
    void* y;
    const int* pos;            // null: token t has row t (dropout alone)
    const float* gates;        // null: 1
    int64_t ldrows, ldadd, ldy;
    uint32_t T, first;         // tokens of this launch: first .. first + T - 1
    uint32_t n_rows;
    int D, k, add_fp32;
    Divisor packs;             // of a row of y
    Dropout drop;
};

// Columns c .. of add_t: of the rows' type, or fp32 beside rows of 16 bits.
template <class T, int HOW>
struct AddCols {
    Cols<T, HOW> v;
    Cols<float, HOW> f[2];
    static __device__ __forceinline__ bool wide(const Gather& a) { return sizeof(T) == 2 && a.add_fp32; }
    __device__ __forceinline__ void load(const Gather& a, uint32_t t, int c) {
        if (!a.add) return;
        if (wide(a)) {
            const float* row = static_cast<const float*>(a.add) + (int64_t)t * a.ldadd;
            f[0].load(row, c, a.D);
            f[1].load(row, c + 4, a.D);
        } else {
            v.load(static_cast<const T*>(a.add) + (int64_t)t * a.ldadd, c, a.D);
        }
    }
    __device__ __forceinline__ void add_to(F2* o, const Gather& a) const {
        if (!a.add) return;
        F2 x[4];
        if (wide(a)) unpack16<float>(f[0].get(), x), unpack16<float>(f[1].get(), x + 2);
        else unpack16<T>(v.get(), x);
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) o[i] = o[i] + x[i];
    }
};

template <class T>
__device__ __forceinline__ void prefetch_add(const Gather& a, uint32_t t, int c) {
    const int64_t at = (int64_t)t * a.ldadd + c;
    const void* p = sizeof(T) == 2 && a.add_fp32 ? static_cast<const void*>(static_cast<const float*>(a.add) + at) : static_cast<const T*>(a.add) + at;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Columns c .. of y_t, AHEAD rows' loads at a time.
template <class T, int HOW, bool DROP, bool SELF, int AHEAD>
__device__ __forceinline__ void gather(const Gather& a, uint32_t t, T* y, int c) {
    constexpr int V2 = kVec<T> / 2;
    const T* rows = static_cast<const T*>(a.rows);
    F2 v[V2];
    AddCols<T, HOW> add;
    if constexpr (SELF) {
        Cols<T, HOW> x;
        x.load(rows + (int64_t)t * a.ldrows, c, a.D);
        add.load(a, t, c);
        unpack16<T>(x.get(), v);
    } else {
#pragma unroll
        for (int i = 0; i < V2; ++i) v[i] = f2(0.f);
        const int64_t pair = (int64_t)t * a.k;
        uint32_t at[AHEAD];
        float g[AHEAD];
        auto load_pairs = [&](int j0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                at[i] = j0 + i < a.k ? (uint32_t)a.pos[pair + j0 + i] : ~0u;
                g[i] = a.gates && j0 + i < a.k ? a.gates[pair + j0 + i] : 1.f;
            }
        };
        load_pairs(0);
        // the sum's last addend is loaded last, when registers are free, out of L2 (8192 tokens' 2 choices of
        // 4096 bf16 columns: 41.5 us, without 44.5)
        if (HOW == kOnPacks && a.add) prefetch_add<T>(a, t, c);
        for (int j0 = 0; j0 < a.k; j0 += AHEAD) {
            Cols<T, HOW> x[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (at[i] < a.n_rows) x[i].load(rows + (int64_t)at[i] * a.ldrows, c, a.D);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (at[i] >= a.n_rows) continue;
                F2 f[V2];
                unpack16<T>(x[i].get(), f);
                const F2 w = f2(g[i]);
#pragma unroll
                for (int q = 0; q < V2; ++q) v[q] = fma(w, f[q], v[q]);
            }
            load_pairs(j0 + AHEAD);
        }
    }
    if constexpr (!SELF) add.load(a, t, c);
    if constexpr (DROP) drop<T>(v, dropout_bits<T, HOW == kOnPacks>(a.drop, dropout_offset(a.drop), t, c), a.drop.keep, a.drop.scale);
    add.add_to(v, a);
    store_cols<T, HOW>(y, c, a.D, pack16<T>(v));
}

// y_t = add_t + drop(sum_j g_tj rows[pos_tj]), a pack of y a thread.  Sums and products in fp32, by rising
// j; the one rounding to fewer bits is y's.
template <class T, Lie LIE, bool DROP, bool SELF>
__device__ __forceinline__ void gather_item(const Gather& a) {
    const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t n = a.packs.quotient(item), t = a.first + n;
    if (n >= a.T) return;
    T* y = static_cast<T*>(a.y) + (int64_t)t * a.ldy;
    const int k = item - n * a.packs.d;
    if constexpr (LIE == kWhole) {
        gather<T, kOnPacks, DROP, SELF, 2>(a, t, y, k * kVec<T>);
    } else if constexpr (LIE == kApart) {
        if (single_col(k) < a.D) gather<T, kSingles, DROP, SELF, 2>(a, t, y, single_col(k));
    } else {
        const int c = first_col(y, k);
        if (c >= a.D) return;
        const bool packs = LIE == kAlike ? c >= 0 && c + kVec<T> <= a.D : a.D >= kVec<T>;
        if (packs) gather<T, LIE == kAlike ? kAligned : kAnywhere, DROP, SELF, 2>(a, t, y, c);
        else gather<T, kElements, DROP, SELF, 1>(a, t, y, c);
    }
}
// (Shifted packs take more registers: 5 CTAs an SM.)
template <class T, Lie LIE, bool DROP>
__global__ void __launch_bounds__(kThreads, LIE == kShifted ? 5 : 8) moe_gather_kernel(const __grid_constant__ Gather a) {
    after_previous();
    gather_item<T, LIE, DROP, false>(a);
}
// Dropout alone: HBM, with 45 % of the issue slots taken (of odd width, rows alike: 55 us for 36 of traffic;
// a thread's columns then lie in two of the generator's blocks).
template <class T, Lie LIE, bool DROP>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ Gather a) {
    after_previous();
    gather_item<T, LIE, DROP, true>(a);
}

// ---------------------------------------------------------------- tokens to rows

struct Scatter {
    const void *x, *rows;      // rows: the experts' outputs (gradient of the combine)
    void* out;
    const int* pos;
    const float* gates;
    float* dgates;
    int64_t ldx, ldrows, ldout;
    uint32_t T, first, n_rows;
    int D, k;
    Divisor packs, top;        // packs of a row; choices of a token
    Dropout drop;
};

// Pack k of each of a token's rows, AHEAD of them at a time.
template <class T, int HOW, int AHEAD>
__device__ __forceinline__ void scatter_packs(const Scatter& a, const int* pos, const T* x, T* out, int k) {
    for (int j0 = 0; j0 < a.k; j0 += AHEAD) {
        uint32_t at[AHEAD];
        int c[AHEAD];
        Cols<T, HOW> v[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) at[i] = j0 + i < a.k ? (uint32_t)pos[j0 + i] : ~0u;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            c[i] = at[i] < a.n_rows ? first_col(out + (int64_t)at[i] * a.ldout, k) : a.D;
            if (c[i] < a.D) v[i].load(x, c[i], a.D);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (c[i] < a.D) store_cols<T, HOW>(out + (int64_t)at[i] * a.ldout, c[i], a.D, v[i].get());
    }
}

// rows[pos_tj] = x_t, a pack of x a thread, read once and written to each of its rows: HBM, 6.5 TB/s;
// kShifted: a pack of each of the token's rows, whose boundaries differ (8192 tokens to 2 of 4095 bf16 columns 41
// us for 30 of traffic, with the sort 44).
template <class T, Lie LIE>
__global__ void __launch_bounds__(kThreads) moe_scatter_kernel(const __grid_constant__ Scatter a) {
    after_previous();
    const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t n = a.packs.quotient(item), t = a.first + n;
    if (n >= a.T) return;
    const int k = item - n * a.packs.d;
    const int* pos = a.pos + (int64_t)t * a.k;
    const T* x = static_cast<const T*>(a.x) + (int64_t)t * a.ldx;
    T* out = static_cast<T*>(a.out);
    if constexpr (LIE != kShifted) {
        constexpr int how = LIE == kWhole ? kOnPacks : kSingles;
        const int c = LIE == kWhole ? k * kVec<T> : single_col(k);
        if (LIE == kApart && c >= a.D) return;
        const uint4 v = load_cols<T, how>(x, c, a.D);
        for (int j = 0; j < a.k; ++j) {
            const uint32_t at = (uint32_t)pos[j];
            if (at < a.n_rows) store_cols<T, how>(out + (int64_t)at * a.ldout, c, a.D, v);
        }
    } else {
        if (a.D >= kVec<T>) scatter_packs<T, kAnywhere, 2>(a, pos, x, out, k);
        else scatter_packs<T, kElements, 1>(a, pos, x, out, k);
    }
}

// Columns c .. of drop(dy_t).
template <class T, int HOW, bool DROP>
__device__ __forceinline__ void dropped_cols(F2* e, const Scatter& a, uint64_t offset, uint32_t t, int c) {
    Cols<T, HOW> d;
    d.load(static_cast<const T*>(a.x) + (int64_t)t * a.ldx, c, a.D);
    uint4 bits;
    if constexpr (DROP) bits = dropout_bits<T, HOW == kOnPacks>(a.drop, offset, t, c);
    unpack16<T>(d.get(), e);
    if constexpr (DROP) drop<T>(e, bits, a.drop.keep, a.drop.scale);
}

// Both halves of a warp's sums at once: lane 0 has v0's, lane 16 v1's.
__device__ __forceinline__ float warp_sums(float v0, float v1) {
    const bool low = (threadIdx.x & 16) == 0;
    float v = (low ? v0 : v1) + __shfl_xor_sync(0xffffffffu, low ? v1 : v0, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The combine's gradient: with e = drop(dy_t), drows[pos_tj] = g_tj e and dgates_tj = <e, rows[pos_tj]>.
// A CTA a token.  Up to CHOICES choices: all of them at a time, their sums in registers, so a token's
// gradient and its dropout are read and computed once (4096 tokens of 6 experts of 2048 bf16, p 0.1: 37 us
// for 32.7 of traffic, two at a time 38.3; the CTAs an SM as they measured best: 8192 tokens of 2, 51 us at 6,
// 52 at 5).
template <class T, Lie LIE, bool DROP, int CHOICES>
__global__ void __launch_bounds__(kThreads, CHOICES == 2 ? 6 : CHOICES == 4 ? 4 : 3) moe_combine_bwd_few_kernel(const __grid_constant__ Scatter a) {
    after_previous();
    constexpr int V2 = kVec<T> / 2, how = LIE == kWhole ? kOnPacks : kSingles;
    __shared__ float part[kThreads / 32][CHOICES];
    const uint32_t t = a.first + blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t pair = (int64_t)t * a.k;
    uint32_t at[CHOICES];
    float g[CHOICES];
    float sum[CHOICES];
#pragma unroll
    for (int i = 0; i < CHOICES; ++i) {
        at[i] = i < a.k ? (uint32_t)a.pos[pair + i] : ~0u;
        g[i] = i < a.k ? a.gates[pair + i] : 0.f;
        sum[i] = 0.f;
    }
    for (int k = threadIdx.x; k < (int)a.packs.d; k += blockDim.x) {
        const int c = LIE == kWhole ? k * kVec<T> : single_col(k);
        if (LIE != kWhole && c >= a.D) break;
        Cols<T, how> d, x[CHOICES];
        d.load(static_cast<const T*>(a.x) + (int64_t)t * a.ldx, c, a.D);
#pragma unroll
        for (int i = 0; i < CHOICES; ++i)
            if (at[i] < a.n_rows) x[i].load(static_cast<const T*>(a.rows) + (int64_t)at[i] * a.ldrows, c, a.D);
        uint4 bits;
        if constexpr (DROP) bits = dropout_bits<T, true>(a.drop, dropout_offset(a.drop), t, c);
        F2 e[V2];
        unpack16<T>(d.get(), e);
        if constexpr (DROP) drop<T>(e, bits, a.drop.keep, a.drop.scale);
#pragma unroll
        for (int i = 0; i < CHOICES; ++i) {
            if (at[i] >= a.n_rows) continue;
            F2 f[V2], s = f2(0.f);
            unpack16<T>(x[i].get(), f);
            const F2 w = f2(g[i]);
#pragma unroll
            for (int q = 0; q < V2; ++q) {
                s = fma(e[q], f[q], s);
                f[q] = w * e[q];
            }
            const float2 p = split(s);
            sum[i] += p.x + p.y;
            store_cols<T, how>(static_cast<T*>(a.out) + (int64_t)at[i] * a.ldout, c, a.D, pack16<T>(f));
        }
    }
#pragma unroll
    for (int i = 0; i < CHOICES; i += 2) {
        const float v = warp_sums(sum[i], sum[i + 1]);
        if ((lane & 15) == 0) part[warp][i + (lane >> 4)] = v;
    }
    __syncthreads();
    if ((int)threadIdx.x < a.k) {
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += part[w][threadIdx.x];
        a.dgates[pair + threadIdx.x] = v;
    }
}

// More choices: two at a time for each pack of dy_t, so that it and its dropout are computed once; `part`: a
// sum a warp for each choice (2048 tokens of 16 of 2048 bf16 columns, dropout: 49 us for 41.5 of traffic).
template <class T, Lie LIE, bool DROP>
__global__ void __launch_bounds__(kThreads, 6) moe_combine_bwd_kernel(const __grid_constant__ Scatter a) {
    after_previous();
    constexpr int V2 = kVec<T> / 2, how = LIE == kWhole ? kOnPacks : kSingles;
    extern __shared__ float part[];        // [top_k][warps]
    const uint32_t t = a.first + blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const T* rows = static_cast<const T*>(a.rows);
    T* drows = static_cast<T*>(a.out);
    const int64_t pair = (int64_t)t * a.k;
    uint64_t offset = 0;
    if constexpr (DROP) offset = dropout_offset(a.drop);
    // every lane takes part in the sums, with a pack or without
    for (int k0 = warp * 32; k0 < (int)a.packs.d; k0 += blockDim.x) {
        const int k = k0 + lane, c = LIE == kWhole ? k * kVec<T> : single_col(k);
        const bool in = LIE == kWhole ? k < (int)a.packs.d : c < a.D;
        F2 e[V2];
        if (in) dropped_cols<T, how, DROP>(e, a, offset, t, c);
        for (int j = 0; j < a.k; j += 2) {
            const uint32_t at0 = (uint32_t)a.pos[pair + j], at1 = j + 1 < a.k ? (uint32_t)a.pos[pair + j + 1] : ~0u;
            const bool in0 = in && at0 < a.n_rows, in1 = in && at1 < a.n_rows;
            Cols<T, how> x0, x1;
            if (in0) x0.load(rows + (int64_t)at0 * a.ldrows, c, a.D);
            if (in1) x1.load(rows + (int64_t)at1 * a.ldrows, c, a.D);
            F2 s0 = f2(0.f), s1 = s0, f[V2];
            auto choice = [&](const Cols<T, how>& x, F2& s, uint32_t at, int at_j) {
                const F2 g = f2(a.gates[pair + at_j]);
                unpack16<T>(x.get(), f);
#pragma unroll
                for (int q = 0; q < V2; ++q) {
                    s = fma(e[q], f[q], s);
                    f[q] = g * e[q];
                }
                store_cols<T, how>(drows + (int64_t)at * a.ldout, c, a.D, pack16<T>(f));
            };
            if (in0) choice(x0, s0, at0, j);
            if (in1) choice(x1, s1, at1, j + 1);
            const float2 p0 = split(s0), p1 = split(s1);
            const float v = warp_sums(p0.x + p0.y, p1.x + p1.y);
            const int mine = j + (lane >> 4);
            if ((lane & 15) == 0 && mine < a.k) {
                float* p = part + mine * warps + warp;
                *p = k0 < (int)blockDim.x ? v : *p + v;
            }
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += part[j * warps + w];
        a.dgates[pair + j] = v;
    }
}

// Rows off 16-byte boundaries differ from row to row, so each choice has packs of its own.  Columns c .. of
// drows = g e, and their part of <e, rows>; drop(e, c) makes e of dy.
template <class T, int HOW, class Drop>
__device__ __forceinline__ float pair_cols(const T* dy, const T* row, T* to, F2 g, int c, int D, const Drop& drop) {
    constexpr int V2 = kVec<T> / 2;
    Cols<T, HOW> x, d;
    x.load(row, c, D);
    d.load(dy, c, D);
    F2 e[V2], f[V2], s = f2(0.f);
    unpack16<T>(d.get(), e);
    drop(e, c);
    unpack16<T>(HOW == kAnywhere && (x.m | x.moved) == 0 ? x.lo : x.get(), f);       // rows that lie as drows do
#pragma unroll
    for (int q = 0; q < V2; ++q) {
        s = fma(e[q], f[q], s);
        f[q] = g * e[q];
    }
    store_cols<T, HOW>(to, c, D, pack16<T>(f));
    const float2 p = split(s);
    return p.x + p.y;
}
// Packs k, k + step, ... below `end` of a choice.
template <class T, class Drop>
__device__ __forceinline__ float pair_packs(const Scatter& a, uint32_t t, uint32_t at, float g, int k, int end, int step, const Drop& drop) {
    const T *dy = static_cast<const T*>(a.x) + (int64_t)t * a.ldx, *row = static_cast<const T*>(a.rows) + (int64_t)at * a.ldrows;
    T* to = static_cast<T*>(a.out) + (int64_t)at * a.ldout;
    float sum = 0.f;
    for (; k < end; k += step) {
        const int c = first_col(to, k);
        if (c >= a.D) break;
        sum += a.D >= kVec<T> ? pair_cols<T, kAnywhere>(dy, row, to, f2(g), c, a.D, drop)
                              : pair_cols<T, kElements>(dy, row, to, f2(g), c, a.D, drop);
    }
    return sum;
}

// Without dropout: `lanes` threads a choice, one warp (four choices a CTA, no barrier) or the CTA.  (A CTA a
// token with a warp a choice, as below: 34 us where this took 27 for 4099 tokens' 7 choices of 1021 columns.)
template <class T>
__global__ void __launch_bounds__(kThreads, 6) moe_combine_bwd_pairs_kernel(const __grid_constant__ Scatter a, int lanes) {
    after_previous();
    __shared__ float part[kThreads / 32];
    const uint32_t p = lanes == 32 ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    const int lane = lanes == 32 ? threadIdx.x & 31 : threadIdx.x;
    const uint32_t n = a.top.quotient(p), t = a.first + n;
    if (n >= a.T) return;                  // a whole warp, of a CTA that has no barrier
    const int64_t pair = (int64_t)t * a.k + (p - n * a.k);
    const uint32_t at = (uint32_t)a.pos[pair];
    float v = 0.f;
    if (at < a.n_rows) v = pair_packs<T>(a, t, at, a.gates[pair], lane, (int)a.packs.d, lanes, [](F2*, int) {});
    v = warp_sum(v);
    if (lanes > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < lanes / 32; ++w) v += part[w];
    }
    if (lane == 0) a.dgates[pair] = v;
}

// With dropout: a CTA a token, `split` warps a choice, kSegment columns at a time, of which it is first
// computed once for all choices, into shared memory, which ones are dropped: a byte for eight columns.
// (Computed at each choice's packs, which begin anywhere in those eight, 2048 tokens' 4 choices of 8191
// bf16 columns took 105 us instead of 71.)
constexpr int kSegment = 32768;
template <class T>
__global__ void __launch_bounds__(kThreads, 6) moe_combine_bwd_drop_kernel(const __grid_constant__ Scatter a, int split) {
    after_previous();
    constexpr int kPacks = kSegment / kVec<T>;
    __shared__ uint8_t keep[kSegment / 8 + 2];             // keep[0]: the eight columns before the segment
    extern __shared__ float part[];                        // [top_k][split]
    const uint32_t t = a.first + blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t pair = (int64_t)t * a.k;
    const uint64_t offset = dropout_offset(a.drop);
    for (int k0 = 0; k0 < (int)a.packs.d; k0 += kPacks) {
        const int c0 = k0 * kVec<T>;
        if (k0 > 0) __syncthreads();
        for (int b = threadIdx.x; b < min(kSegment, a.D - c0 + 7) / 8 + 2; b += blockDim.x)
            keep[b] = dropout_byte(a.drop, offset, t, (uint32_t)(c0 / 8 - 1 + b));
        __syncthreads();
        for (int j = warp / split; j < a.k; j += (blockDim.x >> 5) / split) {
            const uint32_t at = (uint32_t)a.pos[pair + j];
            float sum = 0.f;
            if (at < a.n_rows)
                sum = pair_packs<T>(a, t, at, a.gates[pair + j], k0 + warp % split * 32 + lane, min(k0 + kPacks, (int)a.packs.d),
                                    split * 32, [&](F2* e, int c) {
                                        const uint8_t* bytes = keep + 1 + ((c - c0) >> 3);
                                        drop<T>(e, (uint32_t)(bytes[0] | bytes[1] << 8) >> (c & 7), a.drop.scale);
                                    });
            sum = warp_sum(sum);
            if (lane == 0) {
                float* p = part + j * split + warp % split;
                *p = k0 == 0 ? sum : *p + sum;
            }
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < split; ++w) v += part[j * split + w];
        a.dgates[pair + j] = v;
    }
}

// ---------------------------------------------------------------- host side

struct Rows16 {
    int64_t bits = 0, first = -1;
    bool alike = true;
    void add(const void* p, int64_t ld, int size) {
        if (!p) return;
        const int64_t base = (int64_t)(reinterpret_cast<uintptr_t>(p) & 15), step = ld * size & 15;
        bits |= base | step;
        if (first < 0) first = base << 4 | step;
        alike = alike && first == (base << 4 | step);
    }
    Lie lie(int64_t D, int size, bool dropping, bool self) const {
        if (((bits | (D * size)) & 15) == 0) return kWhole;
        if (size == 4 && !dropping) return kApart;
        return self && alike ? kAlike : kShifted;
    }
};

// Items of an output row, a thread each: packs, of which shifted rows may have one more than they fill (they
// start up to a pack less an element into their first one), or 32 for 128 columns.
uint32_t items_of(int64_t D, int size, Lie lie) {
    const int v = 16 / size;
    return (uint32_t)(lie == kWhole ? D / v : lie == kApart ? (D + 127) / 128 * 32 : (D + 2 * v - 2) / v);
}

// Tokens of a launch, each of `items` threads: kernels number them by 31 bits.
int64_t tokens_of_launch(int64_t T, int64_t items) {
    const int64_t most = std::max<int64_t>(1, ((int64_t(1) << 31) - kThreads) / items);
    return std::min(T, most);
}

// f.go<T, LIE, DROP>() for a call's rows.
template <class F>
struct WithRows {
    const F& f;
    Lie lie;
    bool dropping;
    template <class T>
    cudaError_t run() const {
        if (lie == kWhole) return dropping ? f.template go<T, kWhole, true>() : f.template go<T, kWhole, false>();
        if constexpr (sizeof(T) == 4)
            if (lie == kApart) return f.template go<T, kApart, false>();
        if constexpr (F::kAlikeRows)
            if (lie == kAlike) return dropping ? f.template go<T, kAlike, true>() : f.template go<T, kAlike, false>();
        return dropping ? f.template go<T, kShifted, true>() : f.template go<T, kShifted, false>();
    }
};

struct LaunchGather {
    static constexpr bool kAlikeRows = true;
    const Gather& a;
    cudaStream_t s;
    template <class T, Lie LIE, bool DROP>
    cudaError_t go() const {
        const unsigned grid = (unsigned)(((uint64_t)a.T * a.packs.d + kThreads - 1) / kThreads);
        if constexpr (LIE != kAlike)
            if (a.pos) return launch_early(moe_gather_kernel<T, LIE, DROP>, grid, kThreads, 0, s, a);
        return launch_early(dropout_kernel<T, LIE, DROP>, grid, kThreads, 0, s, a);
    }
};

// A row's place differs from its token's, so no rows are alike below.
struct LaunchScatter {
    static constexpr bool kAlikeRows = false;
    const Scatter& a;
    cudaStream_t s;
    template <class T, Lie LIE, bool>
    cudaError_t go() const {
        const uint64_t items = (uint64_t)a.T * a.packs.d;
        return launch_early(moe_scatter_kernel<T, LIE>, (unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, s, a);
    }
};

struct LaunchCombineBwd {
    static constexpr bool kAlikeRows = false;
    const Scatter& a;
    cudaStream_t s;
    template <class T, Lie LIE, bool DROP>
    cudaError_t go() const {
        const int wide = (int)(a.packs.d + 31) / 32;
        if constexpr (LIE == kShifted && DROP) {   // as many warps a choice as there are for all, and as its packs are for
            int split = 1;
            while (2 * split * a.k <= kThreads / 32 && 2 * split <= wide) split *= 2;
            const int warps = std::min(kThreads / 32, split * a.k);
            return launch_early(moe_combine_bwd_drop_kernel<T>, a.T, warps * 32, (size_t)a.k * split * sizeof(float), s, a, split);
        } else if constexpr (LIE == kShifted) {        // a warp for rows of up to 16 packs a lane
            const uint64_t pairs = (uint64_t)a.T * a.k;
            const int lanes = wide <= 16 ? 32 : kThreads, threads = lanes == 32 ? 128 : kThreads;
            return launch_early(moe_combine_bwd_pairs_kernel<T>, (unsigned)(lanes == 32 ? (pairs + 3) / 4 : pairs), threads, 0, s, a, lanes);
        } else {
            const int warps = std::min(kThreads / 32, wide);
            if (a.k <= 2) return launch_early(moe_combine_bwd_few_kernel<T, LIE, DROP, 2>, a.T, warps * 32, 0, s, a);
            if (a.k <= 4) return launch_early(moe_combine_bwd_few_kernel<T, LIE, DROP, 4>, a.T, warps * 32, 0, s, a);
            if (a.k <= 8) return launch_early(moe_combine_bwd_few_kernel<T, LIE, DROP, 8>, a.T, warps * 32, 0, s, a);
            return launch_early(moe_combine_bwd_kernel<T, LIE, DROP>, a.T, warps * 32, (size_t)warps * a.k * sizeof(float), s, a);
        }
    }
};

swiglu_status tokens_check(int64_t T, int64_t D, int64_t k, int64_t n_rows, int type, const char* sizes, const char* limits,
                           const char* types) {
    if (T < 0 || D <= 0 || k <= 0 || n_rows < 0) return fail(SWIGLU_ERR_INVALID_ARG, sizes);
    if (T >= (int64_t(1) << 31) || n_rows >= (int64_t(1) << 31) || D >= (int64_t(1) << 28) || k > kMaxTop || D * k >= (int64_t(1) << 31))
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, limits);
    if (type_bytes(type) == 0) return fail(SWIGLU_ERR_INVALID_ARG, types);
    return SWIGLU_OK;
}
#define TOKENS_CHECK(name, T, D, k, n_rows, type)                                                    \
    tokens_check(T, D, k, n_rows, type, name ": a size is negative or zero",                         \
                 name ": T, n_rows and D * top_k must stay below 2^31, D below 2^28, top_k up to 1024", name ": unknown type")

// Runs launches of up to 2^31 threads over all tokens.
swiglu_status run_gather(Gather a, int kind, int64_t T, int type, int add_type, bool dropping, cudaStream_t s) {
    int sms;
    swiglu_status rc = device_sms(&sms);
    const int n = type_bytes(type);
    Rows16 v;
    v.add(a.rows, a.ldrows, n), v.add(a.y, a.ldy, n), v.add(a.add, a.ldadd, type_bytes(add_type));
    const Lie lie = v.lie(a.D, n, dropping, a.pos == nullptr);
    a.packs = Divisor::of(items_of(a.D, n, lie));
    a.add_fp32 = add_type == SWIGLU_FP32;
    const int64_t step = tokens_of_launch(T, a.packs.d);
    for (int64_t t = 0; rc == SWIGLU_OK && t < T; t += step) {
        a.first = (uint32_t)t, a.T = (uint32_t)std::min(step, T - t);
        const LaunchGather f{a, s};
        rc = launch_traced(kind, s, [&] { return with_type(type, WithRows<LaunchGather>{f, lie, dropping}); });
    }
    return rc;
}

template <class Launch>
swiglu_status run_scatter(Scatter a, int64_t T, int type, bool dropping, cudaStream_t s) {
    int sms;
    swiglu_status rc = device_sms(&sms);
    const int n = type_bytes(type);
    Rows16 v;
    v.add(a.x, a.ldx, n), v.add(a.rows, a.ldrows, n), v.add(a.out, a.ldout, n);
    const Lie lie = v.lie(a.D, n, dropping, false);
    a.packs = Divisor::of(items_of(a.D, n, lie));
    a.top = Divisor::of((uint32_t)a.k);
    const int64_t step = tokens_of_launch(T, (int64_t)a.packs.d * (lie == kShifted ? a.k : 1));
    for (int64_t t = 0; rc == SWIGLU_OK && t < T; t += step) {
        a.first = (uint32_t)t, a.T = (uint32_t)std::min(step, T - t);
        const Launch f{a, s};
        rc = launch_traced(SWIGLU_KERNEL_MOE_SCATTER, s, [&] { return with_type(type, WithRows<Launch>{f, lie, dropping}); });
    }
    return rc;
}

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

swiglu_status swiglu_moe_dispatch_fwd(const void* x, int64_t ldx, const int32_t* pos, void* rows, int64_t ldrows,
                                      int64_t T, int64_t D, int64_t top_k, int64_t n_rows, int type, void* stream) {
    swiglu_status rc = TOKENS_CHECK("dispatch", T, D, top_k, n_rows, type);
    if (rc != SWIGLU_OK || T == 0 || n_rows == 0) return rc;
    if (!x || !pos || !rows) return fail(SWIGLU_ERR_INVALID_ARG, "dispatch: a required pointer is null");
    if (ldx < D || ldrows < D) return fail(SWIGLU_ERR_INVALID_ARG, "dispatch: a row stride is smaller than the width");
    const size_t n = type_bytes(type);
    if (misaligned(x, n) || misaligned(rows, n) || misaligned(pos, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "dispatch: a pointer is not aligned to its element");
    Scatter a{};
    a.x = x, a.ldx = ldx, a.pos = pos, a.out = rows, a.ldout = ldrows;
    a.D = (int)D, a.k = (int)top_k, a.n_rows = (uint32_t)n_rows;
    return run_scatter<LaunchScatter>(a, T, type, false, static_cast<cudaStream_t>(stream));
}

swiglu_status swiglu_moe_dispatch_bwd(const void* drows, int64_t lddrows, const int32_t* pos, const void* add,
                                      int64_t ldadd, void* dx, int64_t lddx, int64_t T, int64_t D, int64_t top_k,
                                      int64_t n_rows, int type, int add_type, void* stream) {
    swiglu_status rc = TOKENS_CHECK("dispatch", T, D, top_k, n_rows, type);
    if (rc != SWIGLU_OK || T == 0) return rc;
    if ((!drows && n_rows > 0) || !pos || !dx) return fail(SWIGLU_ERR_INVALID_ARG, "dispatch: a required pointer is null");
    if (add && add_type != type && add_type != SWIGLU_FP32)
        return fail(SWIGLU_ERR_INVALID_ARG, "dispatch: add is of neither the rows' type nor fp32");
    if ((n_rows > 0 && lddrows < D) || lddx < D || (add && ldadd < D))
        return fail(SWIGLU_ERR_INVALID_ARG, "dispatch: a row stride is smaller than the width");
    const size_t n = type_bytes(type);
    if (misaligned(drows, n) || misaligned(dx, n) || (add && misaligned(add, type_bytes(add_type))) || misaligned(pos, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "dispatch: a pointer is not aligned to its element");
    if (add == dx && (add_type != type || astride(add, ldadd, dx, lddx, T)))
        return fail(SWIGLU_ERR_INVALID_ARG, "dispatch: dx is in add's place with another type or row stride");
    Gather a{};
    a.rows = drows, a.ldrows = lddrows, a.pos = pos, a.add = add, a.ldadd = ldadd, a.y = dx, a.ldy = lddx;
    a.D = (int)D, a.k = (int)top_k, a.n_rows = (uint32_t)n_rows;
    return run_gather(a, SWIGLU_KERNEL_MOE_GATHER, T, type, add ? add_type : type, false, static_cast<cudaStream_t>(stream));
}

swiglu_status swiglu_moe_combine_fwd(const void* rows, int64_t ldrows, const int32_t* pos, const float* gates,
                                     const void* residual, int64_t ldr, void* y, int64_t ldy, int64_t T, int64_t D,
                                     int64_t top_k, int64_t n_rows, int type, double p, uint64_t seed,
                                     uint64_t offset, const int64_t* step, void* stream) {
    swiglu_status rc = TOKENS_CHECK("combine", T, D, top_k, n_rows, type);
    if (rc != SWIGLU_OK) return rc;
    Gather a{};
    if (!dropout_of(&a.drop, p, seed, offset, step)) return fail(SWIGLU_ERR_INVALID_ARG, "combine: p is not in 0 .. 1");
    if (T == 0) return SWIGLU_OK;
    if ((!rows && n_rows > 0) || !pos || !gates || !y) return fail(SWIGLU_ERR_INVALID_ARG, "combine: a required pointer is null");
    if ((n_rows > 0 && ldrows < D) || ldy < D || (residual && ldr < D))
        return fail(SWIGLU_ERR_INVALID_ARG, "combine: a row stride is smaller than the width");
    const size_t n = type_bytes(type);
    if (misaligned(rows, n) || misaligned(y, n) || misaligned(residual, n) || misaligned(pos, 4) || misaligned(gates, 4) ||
        misaligned(step, 8))
        return fail(SWIGLU_ERR_MISALIGNED, "combine: a pointer is not aligned to its element");
    if (astride(residual, ldr, y, ldy, T)) return fail(SWIGLU_ERR_INVALID_ARG, "combine: y is in the residual's place with another row stride");
    a.rows = rows, a.ldrows = ldrows, a.pos = pos, a.gates = gates, a.add = residual, a.ldadd = ldr, a.y = y, a.ldy = ldy;
    a.D = (int)D, a.k = (int)top_k, a.n_rows = (uint32_t)n_rows;
    return run_gather(a, SWIGLU_KERNEL_MOE_GATHER, T, type, type, a.drop.keep < 65536, static_cast<cudaStream_t>(stream));
}

swiglu_status swiglu_moe_combine_bwd(const void* dy, int64_t lddy, const void* rows, int64_t ldrows,
                                     const int32_t* pos, const float* gates, void* drows, int64_t lddrows,
                                     float* dgates, int64_t T, int64_t D, int64_t top_k, int64_t n_rows, int type,
                                     double p, uint64_t seed, uint64_t offset, const int64_t* step, void* stream) {
    swiglu_status rc = TOKENS_CHECK("combine", T, D, top_k, n_rows, type);
    if (rc != SWIGLU_OK) return rc;
    Scatter a{};
    if (!dropout_of(&a.drop, p, seed, offset, step)) return fail(SWIGLU_ERR_INVALID_ARG, "combine: p is not in 0 .. 1");
    if (T == 0) return SWIGLU_OK;
    if (!dy || (n_rows > 0 && (!rows || !drows)) || !pos || !gates || !dgates)
        return fail(SWIGLU_ERR_INVALID_ARG, "combine: a required pointer is null");
    if (lddy < D || (n_rows > 0 && (ldrows < D || lddrows < D)))
        return fail(SWIGLU_ERR_INVALID_ARG, "combine: a row stride is smaller than the width");
    const size_t n = type_bytes(type);
    if (misaligned(dy, n) || misaligned(rows, n) || misaligned(drows, n) || misaligned(pos, 4) || misaligned(gates, 4) ||
        misaligned(dgates, 4) || misaligned(step, 8))
        return fail(SWIGLU_ERR_MISALIGNED, "combine: a pointer is not aligned to its element");
    a.x = dy, a.ldx = lddy, a.rows = rows, a.ldrows = ldrows, a.pos = pos, a.gates = gates, a.out = drows, a.ldout = lddrows;
    a.dgates = dgates, a.D = (int)D, a.k = (int)top_k, a.n_rows = (uint32_t)n_rows;
    return run_scatter<LaunchCombineBwd>(a, T, type, a.drop.keep < 65536, static_cast<cudaStream_t>(stream));
}

swiglu_status swiglu_mlp_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* y, int64_t ldy,
                                 int64_t M, int64_t D, int type, double p, uint64_t seed, uint64_t offset,
                                 const int64_t* step, void* stream) {
    swiglu_status rc = TOKENS_CHECK("dropout", M, D, 1, 0, type);
    if (rc != SWIGLU_OK) return rc;
    Gather a{};
    if (!dropout_of(&a.drop, p, seed, offset, step)) return fail(SWIGLU_ERR_INVALID_ARG, "dropout: p is not in 0 .. 1");
    if (M == 0) return SWIGLU_OK;
    if (!x || !y) return fail(SWIGLU_ERR_INVALID_ARG, "dropout: a required pointer is null");
    if (ldx < D || ldy < D || (residual && ldr < D))
        return fail(SWIGLU_ERR_INVALID_ARG, "dropout: a row stride is smaller than the width");
    const size_t n = type_bytes(type);
    if (misaligned(x, n) || misaligned(y, n) || misaligned(residual, n) || misaligned(step, 8))
        return fail(SWIGLU_ERR_MISALIGNED, "dropout: a pointer is not aligned to its element");
    if (astride(x, ldx, y, ldy, M) || astride(residual, ldr, y, ldy, M))
        return fail(SWIGLU_ERR_INVALID_ARG, "dropout: y is in x's or the residual's place with another row stride");
    a.rows = x, a.ldrows = ldx, a.add = residual, a.ldadd = ldr, a.y = y, a.ldy = ldy;
    a.D = (int)D, a.k = 1;
    return run_gather(a, SWIGLU_KERNEL_DROPOUT, M, type, type, a.drop.keep < 65536, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
