// moe_tokens.cu -- tokens to their experts' rows and back, with the gates, dropout and the residual
// stream, the gradients of both, and dropout alone (include/swiglu_tokens.h).
#include <algorithm>

#include "dropout.cuh"
#include "swiglu_tokens.h"

namespace swiglu {
namespace {

constexpr int kMaxTop = 1024;
constexpr int kThreads = 256;

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

// kVec<T> columns of add from c on, added to v.
template <class T, bool EDGE>
__device__ __forceinline__ void add_cols(F2* v, const Gather& a, uint32_t t, int c) {
    F2 f[kVec<T> / 2];
    if (sizeof(T) == 2 && a.add_fp32) {
        const float* row = static_cast<const float*>(a.add) + (int64_t)t * a.ldadd;
        unpack16<float>(load_cols<float, EDGE>(row, c, a.D), f);
        if constexpr (sizeof(T) == 2) unpack16<float>(load_cols<float, EDGE>(row, c + 4, a.D), f + 2);
    } else {
        unpack16<T>(load_cols<T, EDGE>(static_cast<const T*>(a.add) + (int64_t)t * a.ldadd, c, a.D), f);
    }
#pragma unroll
    for (int i = 0; i < kVec<T> / 2; ++i) v[i] = v[i] + f[i];
}

// y_t = add_t + drop(sum_j g_tj rows[pos_tj]), a pack of y a thread.
template <class T, bool EDGE, bool DROP, bool SELF>
__global__ void __launch_bounds__(kThreads) moe_gather_kernel(const Gather a) {
    constexpr int V2 = kVec<T> / 2, kAhead = 4;
    const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t n = a.packs.quotient(item), t = a.first + n;
    if (n >= a.T) return;
    T* y = static_cast<T*>(a.y) + (int64_t)t * a.ldy;
    const int c = first_col<T, EDGE>(y, item - n * a.packs.d);
    if (EDGE && c >= a.D) return;
    const T* rows = static_cast<const T*>(a.rows);
    F2 v[V2];
    if constexpr (SELF) {
        unpack16<T>(load_cols<T, EDGE>(rows + (int64_t)t * a.ldrows, c, a.D), v);
    } else {
#pragma unroll
        for (int i = 0; i < V2; ++i) v[i] = f2(0.f);
        const int64_t pair = (int64_t)t * a.k;
        for (int j0 = 0; j0 < a.k; j0 += kAhead) {
            uint32_t at[kAhead];
            uint4 b[kAhead];
            float g[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) at[i] = j0 + i < a.k ? (uint32_t)__ldg(a.pos + pair + j0 + i) : ~0u;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (at[i] >= a.n_rows) continue;
                b[i] = load_cols<T, EDGE>(rows + (int64_t)at[i] * a.ldrows, c, a.D);
                g[i] = a.gates ? __ldg(a.gates + pair + j0 + i) : 1.f;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (at[i] >= a.n_rows) continue;
                F2 f[V2];
                unpack16<T>(b[i], f);
                const F2 w = f2(g[i]);
#pragma unroll
                for (int x = 0; x < V2; ++x) v[x] = fma(w, f[x], v[x]);
            }
        }
    }
    if constexpr (DROP) drop<T>(v, dropout_bits<T, EDGE>(a.drop, dropout_offset(a.drop), t, c), a.drop.keep, a.drop.scale);
    if (a.add) add_cols<T, EDGE>(v, a, t, c);
    store_cols<T, EDGE>(y, c, a.D, pack16<T>(v));
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

// rows[pos_tj] = x_t, a pack of x a thread; EDGE: a pack of a row, whose boundaries differ from row to row.
template <class T, bool EDGE>
__global__ void __launch_bounds__(kThreads) moe_scatter_kernel(const Scatter a) {
    const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t n = a.packs.quotient(item);
    const int k = item - n * a.packs.d;
    T* out = static_cast<T*>(a.out);
    if constexpr (EDGE) {
        const uint32_t m = a.top.quotient(n), t = a.first + m;
        if (m >= a.T) return;
        const uint32_t at = (uint32_t)__ldg(a.pos + (int64_t)t * a.k + (n - m * a.k));
        if (at >= a.n_rows) return;
        T* to = out + (int64_t)at * a.ldout;
        const int c = first_col<T, true>(to, k);
        if (c >= a.D) return;
        store_cols<T, true>(to, c, a.D, load_cols<T, true>(static_cast<const T*>(a.x) + (int64_t)t * a.ldx, c, a.D));
    } else {
        if (n >= a.T) return;
        const uint32_t t = a.first + n;
        const int c = k * kVec<T>;
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + (int64_t)t * a.ldx + c);
        for (int j = 0; j < a.k; ++j) {
            const uint32_t at = (uint32_t)__ldg(a.pos + (int64_t)t * a.k + j);
            if (at < a.n_rows) *reinterpret_cast<uint4*>(out + (int64_t)at * a.ldout + c) = v;
        }
    }
}

// The combine's gradient: with e = drop(dy_t), drows[pos_tj] = g_tj e and dgates_tj = <e, rows[pos_tj]>.
// A CTA a token, kAhead choices at a time (EDGE: one, as their rows' boundaries differ).
template <class T, bool EDGE, bool DROP>
__global__ void __launch_bounds__(kThreads) moe_combine_bwd_kernel(const Scatter a) {
    constexpr int V2 = kVec<T> / 2, kAhead = EDGE ? 1 : 4;
    __shared__ float part[2][kThreads / 32][kAhead];
    const uint32_t t = a.first + blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const T *dy = static_cast<const T*>(a.x) + (int64_t)t * a.ldx, *rows = static_cast<const T*>(a.rows);
    T* drows = static_cast<T*>(a.out);
    const int64_t pair = (int64_t)t * a.k;
    uint64_t offset = 0;
    if constexpr (DROP) offset = dropout_offset(a.drop);
    for (int j0 = 0, buffer = 0; j0 < a.k; j0 += kAhead, buffer ^= 1) {
        uint32_t at[kAhead];
        float g[kAhead];
        F2 sum[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            at[i] = j0 + i < a.k ? (uint32_t)__ldg(a.pos + pair + j0 + i) : ~0u;
            g[i] = at[i] < a.n_rows ? __ldg(a.gates + pair + j0 + i) : 0.f;
            sum[i] = f2(0.f);
        }
        const T* shape = drows + (int64_t)(at[0] < a.n_rows ? at[0] : 0) * a.ldout;    // EDGE: this row's packs
        for (int k = threadIdx.x; k < (int)a.packs.d; k += blockDim.x) {
            const int c = first_col<T, EDGE>(shape, k);
            if (EDGE && (c >= a.D || at[0] >= a.n_rows)) continue;
            F2 e[V2];
            unpack16<T>(load_cols<T, EDGE>(dy, c, a.D), e);
            uint4 b[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (at[i] < a.n_rows) b[i] = load_cols<T, EDGE>(rows + (int64_t)at[i] * a.ldrows, c, a.D);
            if constexpr (DROP) drop<T>(e, dropout_bits<T, EDGE>(a.drop, offset, t, c), a.drop.keep, a.drop.scale);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (at[i] >= a.n_rows) continue;
                F2 f[V2], o[V2];
                unpack16<T>(b[i], f);
                const F2 w = f2(g[i]);
#pragma unroll
                for (int x = 0; x < V2; ++x) {
                    sum[i] = fma(e[x], f[x], sum[i]);
                    o[x] = w * e[x];
                }
                store_cols<T, EDGE>(drows + (int64_t)at[i] * a.ldout, c, a.D, pack16<T>(o));
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float2 s = split(sum[i]);
            const float v = warp_sum(s.x + s.y);
            if (lane == 0) part[buffer][warp][i] = v;
        }
        __syncthreads();                   // a buffer is rewritten after the other one's barrier
        if (threadIdx.x < kAhead && j0 + (int)threadIdx.x < a.k) {
            float v = 0.f;
            for (int w = 0; w < warps; ++w) v += part[buffer][w][threadIdx.x];
            a.dgates[pair + j0 + threadIdx.x] = v;
        }
    }
}

// ---------------------------------------------------------------- host side

// Whether all rows of a call start and end on 16-byte boundaries.
struct Rows16 {
    int64_t bits = 0;
    void add(const void* p, int64_t ld, int size) {
        if (p) bits |= (int64_t)(reinterpret_cast<uintptr_t>(p) & 15) | (ld * size & 15);
    }
    bool whole(int64_t D, int size) const { return ((bits | (D * size)) & 15) == 0; }
};

// Packs of an output row: EDGE rows may start up to a pack less an element into their first one.
uint32_t packs_of(int64_t D, int size, bool whole) {
    const int v = 16 / size;
    return (uint32_t)(whole ? D / v : (D + 2 * v - 2) / v);
}

// Tokens of a launch, each of `items` threads: kernels number them by 31 bits.
int64_t tokens_of_launch(int64_t T, int64_t items) {
    const int64_t most = std::max<int64_t>(1, ((int64_t(1) << 31) - kThreads) / items);
    return std::min(T, most);
}

struct LaunchGather {
    const Gather& a;
    bool whole, dropping;
    cudaStream_t s;
    template <class T, bool EDGE, bool DROP>
    cudaError_t go() const {
        const unsigned grid = (unsigned)(((uint64_t)a.T * a.packs.d + kThreads - 1) / kThreads);
        if (a.pos) moe_gather_kernel<T, EDGE, DROP, false><<<grid, kThreads, 0, s>>>(a);
        else moe_gather_kernel<T, EDGE, DROP, true><<<grid, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    template <class T>
    cudaError_t run() const {
        return whole ? (dropping ? go<T, false, true>() : go<T, false, false>())
                     : (dropping ? go<T, true, true>() : go<T, true, false>());
    }
};

struct LaunchScatter {
    const Scatter& a;
    bool whole, bwd, dropping;
    cudaStream_t s;
    template <class T, bool EDGE>
    cudaError_t go() const {
        if (!bwd) {
            const uint64_t items = (uint64_t)a.T * a.packs.d * (EDGE ? a.k : 1);
            moe_scatter_kernel<T, EDGE><<<(unsigned)((items + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
        } else {
            const int threads = a.packs.d >= kThreads ? kThreads : (int)(a.packs.d + 31) / 32 * 32;
            if (dropping) moe_combine_bwd_kernel<T, EDGE, true><<<a.T, threads, 0, s>>>(a);
            else moe_combine_bwd_kernel<T, EDGE, false><<<a.T, threads, 0, s>>>(a);
        }
        return cudaGetLastError();
    }
    template <class T>
    cudaError_t run() const { return whole ? go<T, false>() : go<T, true>(); }
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
    const bool whole = v.whole(a.D, n);
    a.packs = Divisor::of(packs_of(a.D, n, whole));
    a.add_fp32 = add_type == SWIGLU_FP32;
    const int64_t step = tokens_of_launch(T, a.packs.d);
    for (int64_t t = 0; rc == SWIGLU_OK && t < T; t += step) {
        a.first = (uint32_t)t, a.T = (uint32_t)std::min(step, T - t);
        rc = launch_traced(kind, s, [&] { return with_type(type, LaunchGather{a, whole, dropping, s}); });
    }
    return rc;
}

swiglu_status run_scatter(Scatter a, int64_t T, int type, bool bwd, bool dropping, cudaStream_t s) {
    int sms;
    swiglu_status rc = device_sms(&sms);
    const int n = type_bytes(type);
    Rows16 v;
    v.add(a.x, a.ldx, n), v.add(a.rows, a.ldrows, n), v.add(a.out, a.ldout, n);
    const bool whole = v.whole(a.D, n);
    a.packs = Divisor::of(packs_of(a.D, n, whole));
    a.top = Divisor::of((uint32_t)a.k);
    const int64_t step = bwd ? T : tokens_of_launch(T, (int64_t)a.packs.d * (whole ? 1 : a.k));
    for (int64_t t = 0; rc == SWIGLU_OK && t < T; t += step) {
        a.first = (uint32_t)t, a.T = (uint32_t)std::min(step, T - t);
        rc = launch_traced(SWIGLU_KERNEL_MOE_SCATTER, s,
                           [&] { return with_type(type, LaunchScatter{a, whole, bwd, dropping, s}); });
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
    return run_scatter(a, T, type, false, false, static_cast<cudaStream_t>(stream));
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
    return run_scatter(a, T, type, true, a.drop.keep < 65536, static_cast<cudaStream_t>(stream));
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
    a.rows = x, a.ldrows = ldx, a.add = residual, a.ldadd = ldr, a.y = y, a.ldy = ldy;
    a.D = (int)D, a.k = 1;
    return run_gather(a, SWIGLU_KERNEL_DROPOUT, M, type, type, a.drop.keep < 65536, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
