// layer_norm.cu -- layer norm forward and backward (include/swiglu_ops.h).
//
// Both directions are bound by HBM: a row is read once into registers, its statistics are
// reduced there, and the result is written once.  At the HBM rate an SM has about 40
// instructions a column for all of it, so what a row costs besides its columns has to be
// spread over many of them, and the columns' arithmetic runs in packed pairs: a row belongs
// to a group of `lanes` threads with NV packs of 16 bytes each (pack k = q * lanes + lane of
// the row, q < NV).  Measured, 11136 x 3584 bf16 with the residual stream's sum (forward) or
// gradient (backward), 319 MB either way: forward 53.6 us, 6.0 TB/s; backward 55.9 us, 5.7 TB/s,
// of the 6.78 TB/s of a copy.
//
// Rows that do not start on 16-byte boundaries (odd widths, strides, bases) go element by
// element with constant offsets.  Moving them in aligned 16-byte pieces, shifted together in
// registers, was tried: its shifting, edges and bounds took 66 instructions a column.
#include "../host.h"
#include "convert.cuh"
#include "swiglu_ops.h"

namespace swiglu {
namespace {

constexpr int kPlanSms = 152;      // grids are planned for the GB300, so that the workspace query sees no device
constexpr int kMaxThreads = 512;   // the forms for rows too wide for registers
constexpr int kBwdThreads = 384;

struct NormFwd {
    const void *x, *r, *gamma, *beta;
    void *y, *s;
    float *mean, *rstd;
    int64_t ldx, ldr, ldy, lds, M;
    int D, lanes, gf32;
    float eps;
};

struct NormBwd {
    const void *dy, *s, *gamma, *skip;
    const float *mean, *rstd;
    void* dx;
    float *pg, *pb;                // partial planes [gridDim][D] of dgamma and dbeta (NULL: not wanted)
    int64_t lddy, lds, ldk, lddx, M;
    int D, lanes, gf32;
};

// ---------------------------------------------------------------- 16-byte packs of a row

template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// 16 bytes, of which `bytes` are read and the rest are zero.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes = 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 load_smem(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_async() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row read and the next one in flight, in shared memory, filled by asynchronous copies.  A
// thread copies and reads its own packs, so this needs no barrier.  Layout:
// [tensor][stage][pack][thread].
constexpr int kStages = 2;

template <class T, int NV>
struct Rows {
    const char* next = nullptr;            // this lane's pack 0 of the row to copy
    int64_t hop = 0;                       // bytes from a group's row to its next
    uint32_t slot = 0;                     // shared address of this thread's slot, stage 0, pack 0
    uint32_t per = 0;                      // bytes from a pack's slots to the next pack's
    __device__ __forceinline__ void init(const T* base, int64_t ld, int64_t row, int64_t step, int lane, uint32_t smem,
                                         int tensor) {
        next = reinterpret_cast<const char*>(base + row * ld) + lane * 16;
        hop = step * ld * (int64_t)sizeof(T);
        per = blockDim.x * 16;
        slot = smem + tensor * kStages * NV * per + threadIdx.x * 16;
    }
    // Copies the group's next row into a stage; `lane16`: 16 x lane, `pitch`: 16 x lanes.
    __device__ __forceinline__ void issue(int stage, int lane16, int pitch, int row_bytes) {
        const uint32_t to = slot + stage * NV * per;
#pragma unroll
        for (int q = 0; q < NV; ++q)
            if (q < NV - 1 || q * pitch + lane16 < row_bytes) copy_async(to + q * per, next + q * pitch);
        next += hop;
    }
    // Pack q of a stage, once its copies have landed.
    __device__ __forceinline__ uint4 get(int stage, int q) const { return load_smem(slot + (stage * NV + q) * per); }
};

// gamma as fp32 in shared memory: the first 16 bytes of every pack's values, then
// (16-bit rows) the second 16 bytes of every pack's, so that a warp's 16-byte reads touch
// every bank once.
__host__ __device__ constexpr int padded(int D) { return (D + 7) / 8 * 8; }

template <class T>
__device__ __forceinline__ void stage_param(float* to, const void* p, int gf32, int D, float none) {
    const int half = padded(D) / 2;
    auto put = [&](int c, float v) { to[sizeof(T) == 4 ? c : (c & 4 ? half : 0) + (c >> 3) * 4 + (c & 3)] = v; };
    if (gf32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && p != nullptr && D % 4 == 0) {
#pragma unroll 4
        for (int c = threadIdx.x * 4; c < D; c += blockDim.x * 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + c);
            *reinterpret_cast<uint4*>(&to[sizeof(T) == 4 ? c : (c & 4 ? half : 0) + (c >> 3) * 4]) = v;
        }
        for (int c = D + threadIdx.x; c < padded(D); c += blockDim.x) put(c, 0.f);
        return;
    }
#pragma unroll 8
    for (int c = threadIdx.x; c < padded(D); c += blockDim.x)
        put(c, c >= D ? 0.f : p == nullptr ? none : gf32 ? static_cast<const float*>(p)[c] : to_f32(static_cast<const T*>(p)[c]));
}

// Pack k of one, as pairs.
template <class T>
__device__ __forceinline__ void load_staged(F2* o, uint32_t p, int k, int D) {
    unpack16<float>(load_smem(p + k * 16), o);
    if constexpr (sizeof(T) == 2) unpack16<float>(load_smem(p + padded(D) * 2 + k * 16), o + 2);
}

// One value of gamma or beta.
template <class T>
__device__ __forceinline__ float param(const void* p, int gf32, int col, float none, T*) {
    return p == nullptr ? none : gf32 ? static_cast<const float*>(p)[col] : to_f32(static_cast<const T*>(p)[col]);
}

// Pack k of one from global memory.
template <class T>
__device__ __forceinline__ void load_param16(F2* o, const void* p, int gf32, int k, float none) {
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < kVec<T> / 2; ++i) o[i] = f2(none);
    } else if (sizeof(T) == 2 && gf32) {
        const uint4* q = reinterpret_cast<const uint4*>(p) + 2 * k;
        unpack16<float>(q[0], o);
        unpack16<float>(q[1], o + 2);
    } else {
        unpack16<T>(reinterpret_cast<const uint4*>(p)[k], o);
    }
}

// ---------------------------------------------------------------- sums over a row

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Barrier of a group of threads (barrier 0 is __syncthreads').
__device__ __forceinline__ void group_sync(int group, int lanes) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
}

// Sums over the group's `lanes` threads.  One warp: shuffles.  More: shuffles, then every
// thread adds the warps' sums from shared memory in warp order.  `red`: kRed entries for each
// of two buffers, which the caller alternates, so that one barrier a reduction is enough: a
// buffer is rewritten only after the other one's barrier, which every reader of the first
// has passed.  The entries past the group's warps hold zeros.
constexpr int kRed = 24;

__device__ __forceinline__ float row_sum(float v, int group, int lanes, float* red, int buf) {
    v = warp_sum(v);
    if (lanes == 32) return v;
    red += buf * kRed;
    if ((threadIdx.x & 31) == 0) red[(threadIdx.x - group * lanes) >> 5] = v;
    group_sync(group, lanes);
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kRed; w += 4) {
        if (w * 32 >= lanes) break;
        const float4 f = *reinterpret_cast<const float4*>(red + w);
        v += (f.x + f.y) + (f.z + f.w);
    }
    return v;
}

// Two sums at once.  The first exchange leaves the low half-warp with x and the high half
// with y, so that the two take 5 or 6 shuffles instead of 10.
__device__ __forceinline__ float2 row_sum2(float2 v, int group, int lanes, float2* red, int buf) {
    const bool high = threadIdx.x & 16;
    float t = (high ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, high ? v.x : v.y, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lanes == 32) {
        const float u = __shfl_xor_sync(0xffffffffu, t, 16);
        return high ? make_float2(u, t) : make_float2(t, u);
    }
    red += buf * kRed;
    if ((threadIdx.x & 15) == 0) reinterpret_cast<float*>(&red[(threadIdx.x - group * lanes) >> 5])[high] = t;
    group_sync(group, lanes);
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kRed; w += 2) {
        if (w * 32 >= lanes) break;
        const float4 f = *reinterpret_cast<const float4*>(red + w);
        v.x += f.x + f.z;
        v.y += f.y + f.w;
    }
    return v;
}

// ---------------------------------------------------------------- forward

// Whether pack k = q * lanes + lane is the row's: the plan gives a row ceil(packs / lanes)
// packs a thread, so only the last one can be past it.
template <class T, int NV>
__device__ __forceinline__ bool in_row(int q, int k, int D) {
    return q < NV - 1 || k * kVec<T> < D;
}

// One row for each group of `lanes` threads: a CTA is one row of more than a warp, or four
// rows of one.  Many small CTAs take turns at loading, reducing and storing; a persistent
// form with the next row in flight in shared memory took 57 us where this takes 53
// (11136 x 3584 bf16).  The statistics need one barrier: a warp centres its columns on its
// own mean, and the warps' (mean, sum of squares about it) are joined exactly.
template <class T, int NV, bool RES, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) layer_norm_fwd_kernel(const NormFwd a) {
    constexpr int V = kVec<T>, P = V / 2;
    __shared__ float2 red[THREADS / 32];
    const int lanes = a.lanes, lane = threadIdx.x % lanes, D = a.D;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / lanes) + threadIdx.x / lanes;
    if (row >= a.M) return;                // whole warps; with more than one warp a row, no thread
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row * a.ldx);
    const uint4* r = reinterpret_cast<const uint4*>(static_cast<const T*>(a.r) + row * a.ldr);
    F2 v[NV * P];
    {
        uint4 px[NV], pr[NV];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane;
            px[q] = pr[q] = make_uint4(0, 0, 0, 0);
            if (in_row<T, NV>(q, k, D)) {
                px[q] = __ldcs(x + k);
                if (RES) pr[q] = __ldcs(r + k);
            }
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            F2* w = v + q * P;
            unpack16<T>(px[q], w);
            if (RES) {
                F2 f[P];
                unpack16<T>(pr[q], f);
#pragma unroll
                for (int i = 0; i < P; ++i) w[i] = w[i] + f[i];
            }
        }
    }
    if (RES) {
        uint4* s = reinterpret_cast<uint4*>(static_cast<T*>(a.s) + row * a.lds);
#pragma unroll
        for (int q = 0; q < NV; ++q)
            if (in_row<T, NV>(q, q * lanes + lane, D)) s[q * lanes + lane] = pack16<T>(v + q * P);
    }
    F2 sum2 = f2(0.f);
#pragma unroll
    for (int i = 0; i < NV * P; ++i) sum2 = sum2 + v[i];
    // columns of warp w: of every pack its 32 * V from (q * lanes + 32 w) * V
    auto columns = [&](int w) {
        int n = 0;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int left = D - (q * lanes + 32 * w) * V;
            n += left >= 32 * V ? 32 * V : left > 0 ? left : 0;
        }
        return (float)n;
    };
    const float2 ss = split(sum2);
    const int warp = (threadIdx.x % lanes) >> 5, warps = lanes >> 5;
    float mean = warp_sum(ss.x + ss.y) / columns(warp);
    const F2 mu = f2(-mean);
    F2 sq2 = f2(0.f);
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        if (in_row<T, NV>(q, q * lanes + lane, D)) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const F2 c = v[q * P + i] + mu;
                sq2 = fma(c, c, sq2);
            }
        }
    }
    const float2 qq = split(sq2);
    float sq = warp_sum(qq.x + qq.y);
    if (warps > 1) {
        if ((threadIdx.x & 31) == 0) red[warp] = make_float2(mean, sq);
        __syncthreads();
        float total = 0.f;
        for (int w = 0; w < warps; ++w) total += columns(w) * red[w].x;
        mean = total / (float)D;
        sq = 0.f;
        for (int w = 0; w < warps; ++w) {
            const float d = red[w].x - mean;
            sq += red[w].y + columns(w) * d * d;
        }
    }
    const float rstd = __frsqrt_rn(sq / (float)D + a.eps);
    const F2 rs = f2(rstd), m2 = f2(-mean);
    uint4* y = reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * a.ldy);
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int k = q * lanes + lane;
        if (in_row<T, NV>(q, k, D)) {
            F2 g[P], b[P];
            load_param16<T>(g, a.gamma, a.gf32, k, 1.f);
            load_param16<T>(b, a.beta, a.gf32, k, 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) g[i] = fma((v[q * P + i] + m2) * rs, g[i], b[i]);
            __stcs(y + k, pack16<T>(g));
        }
    }
    if (lane == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
}

// Rows off 16-byte boundaries (odd widths, strides, bases), element by element: thread t of a
// row's THREADS has columns t + i * THREADS, i < kCols, whose offsets are constants; kCols
// loads a thread keep enough bytes in flight, and a warp still reads 64 or 128 bytes in a row.
constexpr int kCols = 16;

template <class T, bool RES, int THREADS>
__global__ void __launch_bounds__(THREADS < 128 ? 128 : THREADS, THREADS > 128 ? 2 : 8)
    layer_norm_fwd_narrow_kernel(const NormFwd a) {
    __shared__ __align__(16) float red[2 * kRed];
    const int t = threadIdx.x % THREADS, D = a.D;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / THREADS) + threadIdx.x / THREADS;
    if (THREADS > 32) {
        if (threadIdx.x < 2 * kRed) red[threadIdx.x] = 0.f;
        __syncthreads();
    }
    if (row >= a.M) return;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx + t;
    const T* r = static_cast<const T*>(a.r) + row * a.ldr + t;
    float v[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        v[i] = 0.f;
        if (t + i * THREADS < D) v[i] = to_f32(x[i * THREADS]);
    }
    if (RES) {
        T* s = static_cast<T*>(a.s) + row * a.lds + t;
#pragma unroll
        for (int i = 0; i < kCols; ++i)
            if (t + i * THREADS < D) v[i] += to_f32(r[i * THREADS]);
#pragma unroll
        for (int i = 0; i < kCols; ++i)
            if (t + i * THREADS < D) s[i * THREADS] = from_f32<T>(v[i]);
    }
    float sum = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) sum += v[i];
    const float mean = row_sum(sum, 0, THREADS, red, 0) / (float)D;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        v[i] -= mean;
        if (t + i * THREADS < D) sq += v[i] * v[i];
    }
    const float rstd = __frsqrt_rn(row_sum(sq, 0, THREADS, red, 1) / (float)D + a.eps);
    T* y = static_cast<T*>(a.y) + row * a.ldy + t;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        if (t + i * THREADS < D) {
            const float g = param(a.gamma, a.gf32, t + i * THREADS, 1.f, (T*)nullptr);
            const float b = param(a.beta, a.gf32, t + i * THREADS, 0.f, (T*)nullptr);
            y[i * THREADS] = from_f32<T>(v[i] * rstd * g + b);
        }
    }
    if (t == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
}

// gamma or beta at column `col`, in the row's type or in fp32 (the forms for wide rows).
template <class T, int VEC>
__device__ __forceinline__ void load_param(float* o, const void* p, int gf32, int col, float none) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = none;
    } else if (gf32) {
        constexpr int V4 = VEC >= 4 ? 4 : 1;
#pragma unroll
        for (int q = 0; q < VEC / V4; ++q)
            load_pack<float, V4>(static_cast<const float*>(p) + col + q * V4).unpack(o + q * V4);
    } else {
        load_pack<T, VEC>(static_cast<const T*>(p) + col).unpack(o);
    }
}

// A row wider than the registers hold: three passes over it, the last two from L2.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_fwd_wide_kernel(const NormFwd a) {
    __shared__ __align__(16) float red[2 * kRed];
    if (threadIdx.x < 2 * kRed) red[threadIdx.x] = 0.f;
    __syncthreads();
    const float inv = 1.f / (float)a.D;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* r = a.r ? static_cast<const T*>(a.r) + row * a.ldr : nullptr;
        auto load = [&](int col, float* v) {
            load_pack<T, VEC>(x + col).unpack(v);
            if (r) {
                float e[VEC];
                load_pack<T, VEC>(r + col).unpack(e);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] += e[j];
            }
        };
        const int first = threadIdx.x * VEC, hop = blockDim.x * VEC;
        float v[VEC], sum = 0.f, sq = 0.f;
        for (int64_t c = first; c < a.D; c += hop) {
            load((int)c, v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += v[j];
            if (r) store_pack<T, VEC>(static_cast<T*>(a.s) + row * a.lds + c, v);
        }
        const float mean = row_sum(sum, 0, blockDim.x, red, 0) * inv;
        for (int64_t c = first; c < a.D; c += hop) {
            load((int)c, v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sq += (v[j] - mean) * (v[j] - mean);
        }
        const float rstd = __frsqrt_rn(row_sum(sq, 0, blockDim.x, red, 1) * inv + a.eps);
        for (int64_t c = first; c < a.D; c += hop) {
            float g[VEC], b[VEC];
            load((int)c, v);
            load_param<T, VEC>(g, a.gamma, a.gf32, (int)c, 1.f);
            load_param<T, VEC>(b, a.beta, a.gf32, (int)c, 0.f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = (v[j] - mean) * rstd * g[j] + b[j];
            store_pack<T, VEC>(static_cast<T*>(a.y) + row * a.ldy + c, v);
        }
        if (threadIdx.x == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

// ---------------------------------------------------------------- backward

// The row's two sums, dx, and fp32 column sums of dy * xh and dy over the group's rows, kept
// in registers; the CTA's groups are added in shared memory at the end and written once, as
// this CTA's partial planes.  A row is read from the ring twice, before and after the
// reduction, which costs less than keeping xh and g beside the column sums.  (With one row
// ahead in registers instead of the ring it took 92 us of 11136 x 3584 bf16.)
// xh = s * rstd - mean * rstd, and
// dx = g * rstd + s * A + B with A = -c2 * rstd^2, B = c2 * mean * rstd^2 - c1 * rstd.
// Shared memory: red [groups][2][kRed] pairs, gamma (whole packs, fp32), then the rows in
// flight, and after them the groups' column sums in their place.
template <class T, int NV, bool SKIP>
__global__ void __launch_bounds__(kBwdThreads) layer_norm_bwd_kernel(const NormBwd a) {
    constexpr int V = kVec<T>, P = V / 2;
    extern __shared__ uint4 smem[];
    const int lanes = a.lanes, lane = threadIdx.x % lanes, group = threadIdx.x / lanes, D = a.D;
    const int rows = blockDim.x / lanes;
    float2* red = reinterpret_cast<float2*>(smem) + group * 2 * kRed;
    float* gamma = reinterpret_cast<float*>(smem) + rows * 4 * kRed;
    float* acc = gamma + padded(D);
    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t row = (int64_t)blockIdx.x * rows + group;
    const int lane16 = lane * 16, pitch = lanes * 16, row_bytes = D * (int)sizeof(T);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(acc);
    Rows<T, NV> dy, s, skip;
    dy.init(static_cast<const T*>(a.dy), a.lddy, row, step, lane, ring, 0);
    s.init(static_cast<const T*>(a.s), a.lds, row, step, lane, ring, 1);
    if (SKIP) skip.init(static_cast<const T*>(a.skip), a.ldk, row, step, lane, ring, 2);
    auto issue = [&](int stage, int64_t i) {
        if (i < a.M) {
            dy.issue(stage, lane16, pitch, row_bytes);
            s.issue(stage, lane16, pitch, row_bytes);
            if (SKIP) skip.issue(stage, lane16, pitch, row_bytes);
        }
        commit_async();
    };
    cudaTriggerProgrammaticLaunchCompletion();             // the parameters' kernel may come up meanwhile
    issue(0, row);
    for (int i = threadIdx.x; i < rows * 4 * kRed; i += blockDim.x) reinterpret_cast<float*>(smem)[i] = 0.f;
    stage_param<T>(gamma, a.gamma, a.gf32, D, 1.f);
    const uint32_t gamma_at = (uint32_t)__cvta_generic_to_shared(gamma);
    __syncthreads();
    F2 dg[NV * P], db[NV * P];
#pragma unroll
    for (int i = 0; i < NV * P; ++i) dg[i] = db[i] = f2(0.f);
    float mean = 0.f, rstd = 0.f;
    if (row < a.M) mean = a.mean[row], rstd = a.rstd[row];
    const float inv = 1.f / (float)D;
    for (int stage = 0; row < a.M; row += step, stage ^= 1) {
        issue(stage ^ 1, row + step);
        const float mu = mean, rs = rstd;
        if (row + step < a.M) mean = a.mean[row + step], rstd = a.rstd[row + step];
        wait_async<1>();
        const F2 rs2 = f2(rs), shift = f2(-mu * rs);
        F2 c1 = f2(0.f), c2 = f2(0.f);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane;
            if (in_row<T, NV>(q, k, D)) {
                F2 w[P], d[P], xs[P];
                load_staged<T>(w, gamma_at, k, D);
                unpack16<T>(dy.get(stage, q), d);
                unpack16<T>(s.get(stage, q), xs);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const F2 xh = fma(xs[i], rs2, shift), g = d[i] * w[i];
                    dg[q * P + i] = fma(d[i], xh, dg[q * P + i]);
                    db[q * P + i] = db[q * P + i] + d[i];
                    c1 = c1 + g;
                    c2 = fma(g, xh, c2);
                }
            }
        }
        const float2 p1 = split(c1), p2 = split(c2);
        float2 c = row_sum2(make_float2(p1.x + p1.y, p2.x + p2.y), group, lanes, red, stage);
        c.x *= inv * rs;
        c.y *= inv * rs;
        const F2 A = f2(-c.y * rs), B = f2(c.y * mu * rs - c.x);
        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + row * a.lddx);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane;
            if (in_row<T, NV>(q, k, D)) {
                F2 w[P], d[P], xs[P];
                load_staged<T>(w, gamma_at, k, D);
                unpack16<T>(dy.get(stage, q), d);
                unpack16<T>(s.get(stage, q), xs);
#pragma unroll
                for (int i = 0; i < P; ++i) w[i] = fma(d[i] * w[i], rs2, fma(xs[i], A, B));
                if (SKIP) {
                    unpack16<T>(skip.get(stage, q), d);
#pragma unroll
                    for (int i = 0; i < P; ++i) w[i] = w[i] + d[i];
                }
                o[k] = pack16<T>(w);
            }
        }
    }
    if (a.pg == nullptr && a.pb == nullptr) return;
    // the groups' sums meet in the ring's place: [group][2][columns, 16-byte pieces of packs apart]
    wait_async<0>();
    __syncthreads();
    const int width = padded(D), half = sizeof(T) == 2 ? width / 2 : 0;
    float* mine = acc + group * 2 * width;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int k = q * lanes + lane;
        if (in_row<T, NV>(q, k, D)) {
#pragma unroll
            for (int h = 0; h < P / 2; ++h) {
                const float2 g0 = split(dg[q * P + 2 * h]), g1 = split(dg[q * P + 2 * h + 1]);
                const float2 b0 = split(db[q * P + 2 * h]), b1 = split(db[q * P + 2 * h + 1]);
                reinterpret_cast<float4*>(mine + h * half)[k] = make_float4(g0.x, g0.y, g1.x, g1.y);
                reinterpret_cast<float4*>(mine + width + h * half)[k] = make_float4(b0.x, b0.y, b1.x, b1.y);
            }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        const float* p = acc + (sizeof(T) == 4 ? c : (c & 4 ? half : 0) + (c >> 3) * 4 + (c & 3));
        float g = 0.f, b = 0.f;
        for (int w = 0; w < rows; ++w, p += 2 * width) g += p[0], b += p[width];
        if (a.pg) a.pg[(int64_t)blockIdx.x * D + c] = g;
        if (a.pb) a.pb[(int64_t)blockIdx.x * D + c] = b;
    }
}

// Rows off 16-byte boundaries: THREADS threads walk the rows of a worker (a warp, or the CTA),
// whose column sums are its own partial plane.  A row comes to shared memory in the aligned
// 16-byte pieces that cover it, one row ahead, and is read there element by element (loaded
// to registers instead, 2 bytes at a time, it took 207 us where this takes 85 for
// 4864 x 5003 bf16).  Shared memory: [worker][stage][tensor][pitch bytes].
__host__ __device__ constexpr int narrow_pitch(int row_bytes) { return (row_bytes + 14) / 16 * 16 + 16; }

template <class T>
__device__ __forceinline__ void copy_row(char* to, const T* base, int64_t ld, int64_t i, int64_t M, int D, int t, int threads) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base), hi = lo + (uintptr_t)((M - 1) * ld + D) * sizeof(T);
    const uintptr_t start = lo + (uintptr_t)(i * ld) * sizeof(T), first = start & ~uintptr_t(15);
    const int pieces = (int)((start + (uintptr_t)D * sizeof(T) - first + 15) / 16);
    for (int p = t; p < pieces; p += threads) {
        const uintptr_t from = first + (uintptr_t)p * 16;
        char* dst = to + p * 16;
        if (from >= lo) {
            copy_async((uint32_t)__cvta_generic_to_shared(dst), reinterpret_cast<const void*>(from),
                       from + 16 <= hi ? 16 : (int)(hi - from));
        } else {                           // the tensor starts inside this piece
            for (uintptr_t e = lo; e < from + 16 && e < hi; e += sizeof(T))
                *reinterpret_cast<T*>(dst + (e - from)) = *reinterpret_cast<const T*>(e);
        }
    }
}

template <class T, bool SKIP, int THREADS>
__global__ void __launch_bounds__(THREADS < 128 ? 128 : THREADS, THREADS > 128 ? 1 : 4)
    layer_norm_bwd_narrow_kernel(const NormBwd a) {
    constexpr int TENSORS = SKIP ? 3 : 2;
    __shared__ __align__(16) float2 red[2 * kRed];
    extern __shared__ uint4 smem[];
    const int t = threadIdx.x % THREADS, D = a.D, pitch = narrow_pitch(D * (int)sizeof(T));
    const int64_t worker = (int64_t)blockIdx.x * (blockDim.x / THREADS) + threadIdx.x / THREADS;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / THREADS);
    char* rows = reinterpret_cast<char*>(smem) + threadIdx.x / THREADS * 2 * TENSORS * pitch;
    cudaTriggerProgrammaticLaunchCompletion();
    if (THREADS > 32) {
        if (threadIdx.x < 2 * kRed) red[threadIdx.x] = make_float2(0.f, 0.f);
    }
    const T* src[3] = {static_cast<const T*>(a.dy), static_cast<const T*>(a.s), static_cast<const T*>(a.skip)};
    const int64_t ld[3] = {a.lddy, a.lds, a.ldk};
    auto issue = [&](int stage, int64_t i) {
        if (i < a.M) {
#pragma unroll
            for (int k = 0; k < TENSORS; ++k)
                copy_row<T>(rows + (stage * TENSORS + k) * pitch, src[k], ld[k], i, a.M, D, t, THREADS);
        }
        commit_async();
    };
    // this thread's first element of a tensor's row in a stage
    auto at = [&](int stage, int k, int64_t i) {
        const int m = (int)(reinterpret_cast<uintptr_t>(src[k] + i * ld[k]) & 15);
        return reinterpret_cast<const T*>(rows + (stage * TENSORS + k) * pitch + m) + t;
    };
    float dg[kCols], db[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) dg[j] = db[j] = 0.f;
    int64_t row = worker;
    issue(0, row);
    const float inv = 1.f / (float)D;
    for (int stage = 0; row < a.M; row += step, stage ^= 1) {
        const float mu = a.mean[row], rs = a.rstd[row];
        wait_async<0>();
        if (THREADS > 32) group_sync(0, THREADS);          // all pieces are here, and the other stage has been read
        else __syncwarp();
        issue(stage ^ 1, row + step);
        const T *y = at(stage, 0, row), *s = at(stage, 1, row);
        float g[kCols], xh[kCols];
        float2 c = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            if (t + j * THREADS < D) {
                const float d = to_f32(y[j * THREADS]);
                xh[j] = (to_f32(s[j * THREADS]) - mu) * rs;
                g[j] = d * param(a.gamma, a.gf32, t + j * THREADS, 1.f, (T*)nullptr);
                dg[j] += d * xh[j];
                db[j] += d;
                c.x += g[j];
                c.y += g[j] * xh[j];
            }
        }
        c = row_sum2(c, 0, THREADS, red, stage);
        c.x *= inv;
        c.y *= inv;
        T* o = static_cast<T*>(a.dx) + row * a.lddx + t;
        const T* k = at(stage, SKIP ? 2 : 0, row);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            if (t + j * THREADS < D) {
                float v = rs * (g[j] - c.x - xh[j] * c.y);
                if (SKIP) v += to_f32(k[j * THREADS]);
                o[j * THREADS] = from_f32<T>(v);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        if (t + j * THREADS < D) {
            if (a.pg) a.pg[worker * D + t + j * THREADS] = dg[j];
            if (a.pb) a.pb[worker * D + t + j * THREADS] = db[j];
        }
    }
}

// Rows wider than the registers hold, in two passes: the two sums of every row, then dx
// and the column sums of a block of columns over a range of rows.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_bwd_wide_sums_kernel(const NormBwd a, float2* sums) {
    __shared__ __align__(16) float2 red[2 * kRed];
    if (threadIdx.x < 2 * kRed) red[threadIdx.x] = make_float2(0.f, 0.f);
    __syncthreads();
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, buf ^= 1) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const T* s = static_cast<const T*>(a.s) + row * a.lds;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float2 c = make_float2(0.f, 0.f);
        for (int64_t col = threadIdx.x * VEC; col < a.D; col += blockDim.x * VEC) {
            float w[VEC], d[VEC], xs[VEC];
            load_pack<T, VEC>(dy + col).unpack(d);
            load_pack<T, VEC>(s + col).unpack(xs);
            load_param<T, VEC>(w, a.gamma, a.gf32, (int)col, 1.f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = d[j] * w[j];
                c.x += g;
                c.y += g * ((xs[j] - mean) * rstd);
            }
        }
        c = row_sum2(c, 0, blockDim.x, red, buf);
        if (threadIdx.x == 0) sums[row] = make_float2(c.x / (float)a.D, c.y / (float)a.D);
    }
}

// grid (column blocks, row ranges): CTA (x, y) has columns x * blockDim * VEC ... and rows
// y, y + gridDim.y, ...; its column sums are partial plane y.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_bwd_wide_kernel(const NormBwd a, const float2* sums) {
    cudaTriggerProgrammaticLaunchCompletion();
    const int64_t col = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (col >= a.D) return;
    float w[VEC], dg[VEC], db[VEC];
    load_param<T, VEC>(w, a.gamma, a.gf32, (int)col, 1.f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[j] = db[j] = 0.f;
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
        float d[VEC], xs[VEC];
        load_pack<T, VEC>(static_cast<const T*>(a.dy) + row * a.lddy + col).unpack(d);
        load_pack<T, VEC>(static_cast<const T*>(a.s) + row * a.lds + col).unpack(xs);
        const float mean = a.mean[row], rstd = a.rstd[row];
        const float2 c = sums[row];
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float xh = (xs[j] - mean) * rstd;
            dg[j] += d[j] * xh;
            db[j] += d[j];
            o[j] = rstd * (d[j] * w[j] - c.x - xh * c.y);
        }
        if (a.skip) {
            load_pack<T, VEC>(static_cast<const T*>(a.skip) + row * a.ldk + col).unpack(d);
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] += d[j];
        }
        store_pack<T, VEC>(static_cast<T*>(a.dx) + row * a.lddx + col, o);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        if (a.pg) a.pg[(int64_t)blockIdx.y * a.D + col + j] = dg[j];
        if (a.pb) a.pb[(int64_t)blockIdx.y * a.D + col + j] = db[j];
    }
}

// dgamma and dbeta: the planes added in plane order (16 strided runs, then the runs).
template <class W>
__global__ void __launch_bounds__(512) layer_norm_params_kernel(const float* pg, const float* pb, W* dgamma, W* dbeta,
                                                                int planes, int D) {
    __shared__ float part[16][33];
    const float* p = blockIdx.y == 0 ? pg : pb;
    W* out = blockIdx.y == 0 ? dgamma : dbeta;
    if (out == nullptr) return;
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float t = 0.f;
    cudaGridDependencySynchronize();       // launched beside the kernel that writes the planes
    if (col < D) {
#pragma unroll 10
        for (int i = threadIdx.y; i < planes; i += 16) t += p[(int64_t)i * D + col];
    }
    part[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && col < D) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) v += part[w][threadIdx.x];
        out[col] = from_f32<W>(v);
    }
}

// ---------------------------------------------------------------- host side

// How a launch covers its rows: `nv` packs a thread, `lanes` threads a row, `groups` rows a
// CTA at a time.
struct NormPlan {
    int nv, lanes, groups;
    int threads() const { return lanes * groups; }
};

// Packs a thread holds at most.  Backward: the two sums of a pack's columns take 16 registers
// (fp32: 8), and 384 threads have 168 each (11136 x 3584 bf16: 64 us with 512 threads and
// spills, 55.5 with 384, 60.6 with 256; 768 threads of 2 packs: 68.7).
constexpr int kFwdPacks = 4, kBwdPacks = 4;
constexpr size_t kSmem = 227 * 1024;

size_t row_smem(const NormPlan& p, int tensors) { return (size_t)kStages * tensors * p.nv * p.threads() * 16; }
size_t bwd_smem(const NormPlan& p, int64_t D, bool skip) {
    const size_t rows = row_smem(p, skip ? 3 : 2), sums = (size_t)p.groups * 2 * padded((int)D) * 4;
    return (size_t)p.groups * 4 * kRed * 4 + (size_t)padded((int)D) * 4 + (rows > sums ? rows : sums);
}

NormPlan norm_plan(int64_t D, int size, int packs, int threads) {
    NormPlan p;
    const int64_t all = (D * size + 15) / 16;
    p.lanes = (int)((all + packs * 32 - 1) / (packs * 32) * 32);
    p.nv = (int)((all + p.lanes - 1) / p.lanes);
    p.groups = threads / p.lanes > 1 ? threads / p.lanes : 1;
    return p;
}

// Forward: CTAs of one row of more than a warp, or of four rows of one.
NormPlan fwd_plan(int64_t D, int size) {
    NormPlan p = norm_plan(D, size, kFwdPacks, 128);
    if (p.lanes > 32) p.groups = 1;
    return p;
}

// Backward: one CTA on each SM, of as many groups as threads, named barriers and shared
// memory allow, but one row for each SM before two for one.
NormPlan bwd_plan(int64_t M, int64_t D, int size, bool skip) {
    NormPlan p = norm_plan(D, size, kBwdPacks, kBwdThreads);
    if (p.groups > 15) p.groups = 15;                      // barriers 1 .. 15
    const int64_t spread = (M + kPlanSms - 1) / kPlanSms;
    if (spread < p.groups) p.groups = spread > 0 ? (int)spread : 1;
    while (p.groups > 1 && bwd_smem(p, D, skip) > kSmem) --p.groups;
    return p;
}
int bwd_ctas(int64_t M, const NormPlan& p) {
    const int64_t want = (M + p.groups - 1) / p.groups;
    return (int)(want < kPlanSms ? want : kPlanSms);
}

// Widest rows these forms take, by the backward's shared memory: 24 KB, that is 12288 columns
// of 16 bits.
constexpr int64_t kMaxRowBytes = 384 * kBwdPacks * 16;

// Rows element by element: THREADS of a row, and (backward) workers that share the rows; each
// worker has a partial plane, so the wider the row, the fewer.  Wider than 8192: two passes.
int narrow_threads(int64_t D) { return D <= 32 * kCols ? 32 : D <= 128 * kCols ? 128 : 512; }
constexpr int64_t kNarrowWidth = 512 * kCols;
int64_t narrow_workers(int64_t M, int64_t D) {
    const int64_t most = kPlanSms * (int64_t)(narrow_threads(D) == 32 ? 16 : narrow_threads(D) == 128 ? 4 : 1);
    return M < most ? M : most;
}

int64_t wide_row_ranges(int64_t M, int64_t D, int vec) {
    const int64_t blocks = (D + 256 * vec - 1) / (256 * vec);
    int64_t r = (kPlanSms * 8 + blocks - 1) / blocks;
    if (r > 65535) r = 65535;
    return r < M ? r : M;
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// Bytes an element of `type` takes; 0 for an unknown type.
int type_bytes(int type) { return type == SWIGLU_FP32 ? 4 : type == SWIGLU_BF16 || type == SWIGLU_FP16 ? 2 : 0; }

bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// Whether every base, row stride and the width allow 16-byte accesses.
struct Aligned {
    int size, bits = 0;
    void add(const void* p, int64_t ld) {
        if (p) bits |= (int)(reinterpret_cast<uintptr_t>(p) & 15) | (int)((ld * size) & 15);
    }
    bool ok() const { return bits == 0; }
};

// f.run<T>() for the run-time type.
template <class F>
cudaError_t with_type(int type, const F& f) {
    if (type == SWIGLU_FP32) return f.template run<float>();
    if (type == SWIGLU_FP16) return f.template run<__half>();
    return f.template run<__nv_bfloat16>();
}

template <class K>
cudaError_t allow_smem(K kern, size_t bytes) {
    return bytes <= 48 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

struct LaunchFwd {
    const NormFwd& a;
    const NormPlan& p;
    bool shift;                            // rows off 16-byte boundaries
    cudaStream_t s;
    template <class T, int NV, bool RES>
    cudaError_t go() const {
        // 64 registers for the small CTAs, whose number hides the latencies; the larger ones
        // all hold 4 packs a thread
        auto kern = layer_norm_fwd_kernel<T, NV, RES, 128, 8>;
        if constexpr (NV == 4) {
            if (p.threads() > 128) kern = layer_norm_fwd_kernel<T, NV, RES, 384, 2>;
        }
        kern<<<(unsigned)((a.M + p.groups - 1) / p.groups), p.threads(), 0, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int NV>
    cudaError_t res() const {
        return a.r ? go<T, NV, true>() : go<T, NV, false>();
    }
    template <class T, int THREADS>
    cudaError_t narrow() const {
        constexpr int rows = THREADS == 32 ? 4 : 1;
        auto kern = a.r ? layer_norm_fwd_narrow_kernel<T, true, THREADS> : layer_norm_fwd_narrow_kernel<T, false, THREADS>;
        kern<<<(unsigned)((a.M + rows - 1) / rows), THREADS * rows, 0, s>>>(a);
        return cudaGetLastError();
    }
    template <class T>
    cudaError_t run() const {
        if (shift ? a.D > kNarrowWidth : (int64_t)a.D * (int)sizeof(T) > kMaxRowBytes) {
            const unsigned grid = (unsigned)(a.M < kPlanSms * 4 ? a.M : kPlanSms * 4);
            if (shift) layer_norm_fwd_wide_kernel<T, 1><<<grid, kMaxThreads, 0, s>>>(a);
            else layer_norm_fwd_wide_kernel<T, kVec<T>><<<grid, kMaxThreads, 0, s>>>(a);
            return cudaGetLastError();
        }
        if (shift) {
            const int n = narrow_threads(a.D);
            return n == 32 ? narrow<T, 32>() : n == 128 ? narrow<T, 128>() : narrow<T, 512>();
        }
        return p.nv == 1 ? res<T, 1>() : p.nv == 2 ? res<T, 2>() : p.nv == 3 ? res<T, 3>() : res<T, 4>();
    }
};

struct LaunchBwd {
    const NormBwd& a;
    const NormPlan& p;
    bool shift;                            // rows off 16-byte boundaries
    float2* sums;
    int planes;
    cudaStream_t s;
    template <class T, int NV, bool SKIP>
    cudaError_t go() const {
        auto kern = layer_norm_bwd_kernel<T, NV, SKIP>;
        const size_t smem = bwd_smem(p, a.D, SKIP);
        cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)planes, p.threads(), smem, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int NV>
    cudaError_t res() const {
        return a.skip ? go<T, NV, true>() : go<T, NV, false>();
    }
    template <class T, int THREADS>
    cudaError_t narrow() const {
        constexpr int rows = THREADS == 32 ? 4 : 1;
        auto kern = a.skip ? layer_norm_bwd_narrow_kernel<T, true, THREADS> : layer_norm_bwd_narrow_kernel<T, false, THREADS>;
        const size_t smem = (size_t)rows * 2 * (a.skip ? 3 : 2) * narrow_pitch(a.D * (int)sizeof(T));
        cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)(planes / rows), THREADS * rows, smem, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int VEC>
    cudaError_t wide() const {
        const int64_t grid = a.M < kPlanSms * 4 ? a.M : kPlanSms * 4;
        layer_norm_bwd_wide_sums_kernel<T, VEC><<<(unsigned)grid, kMaxThreads, 0, s>>>(a, sums);
        const dim3 tiles((unsigned)((a.D + 256 * VEC - 1) / (256 * VEC)), (unsigned)planes);
        layer_norm_bwd_wide_kernel<T, VEC><<<tiles, 256, 0, s>>>(a, sums);
        return cudaGetLastError();
    }
    template <class T>
    cudaError_t run() const {
        if (shift && a.D > kNarrowWidth) return wide<T, 1>();
        if (!shift && (int64_t)a.D * (int)sizeof(T) > kMaxRowBytes) return wide<T, kVec<T>>();
        if (shift) {
            const int n = narrow_threads(a.D);
            return n == 32 ? narrow<T, 32>() : n == 128 ? narrow<T, 128>() : narrow<T, 512>();
        }
        return p.nv == 1 ? res<T, 1>() : p.nv == 2 ? res<T, 2>() : p.nv == 3 ? res<T, 3>() : res<T, 4>();
    }
};

swiglu_status norm_check(int64_t M, int64_t D, int type, int param_type) {
    if (M < 0 || D <= 0) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a size is negative or zero");
    if (M >= (int64_t(1) << 31) || D >= (int64_t(1) << 28))
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "layer norm: M must stay below 2^31 and D below 2^28");
    if (type_bytes(type) == 0 || (param_type != type && param_type != SWIGLU_FP32))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: unknown type, or parameters of neither the rows' type nor fp32");
    return SWIGLU_OK;
}

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

swiglu_status swiglu_mlp_layer_norm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                        const void* gamma, const void* beta, void* y, int64_t ldy, void* s,
                                        int64_t lds, float* mean, float* rstd, int64_t M, int64_t D, float eps,
                                        int type, int param_type, void* stream) {
    swiglu_status rc = norm_check(M, D, type, param_type);
    if (rc != SWIGLU_OK) return rc;
    if (!(eps >= 0.f)) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: eps is negative");
    if (M == 0) return SWIGLU_OK;
    if (!x || !y) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a required pointer is null");
    if ((residual == nullptr) != (s == nullptr) || (mean == nullptr) != (rstd == nullptr))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: residual and s, and mean and rstd, go together");
    if (ldx < D || ldy < D || (residual && (ldr < D || lds < D)))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a row stride is smaller than the width");
    const size_t n = type_bytes(type), np = type_bytes(param_type);
    if (misaligned(x, n) || misaligned(y, n) || misaligned(residual, n) || misaligned(s, n) || misaligned(gamma, np) ||
        misaligned(beta, np) || misaligned(mean, 4) || misaligned(rstd, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "layer norm: a pointer is not aligned to its element");
    int sms;
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    Aligned v{(int)n};
    v.add(x, ldx), v.add(residual, ldr), v.add(y, ldy), v.add(s, lds), v.add(x, D);
    v.add(gamma, 0), v.add(beta, 0);
    const NormPlan p = fwd_plan(D, (int)n);
    const NormFwd a{x, residual, gamma, beta, y, s, mean, rstd, ldx, ldr, ldy, lds, M, (int)D, p.lanes,
                    param_type == SWIGLU_FP32, eps};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_NORM_FWD, st, [&] { return with_type(type, LaunchFwd{a, p, !v.ok(), st}); });
}

size_t swiglu_mlp_layer_norm_bwd_workspace_size(int64_t M, int64_t D) {
    if (M <= 0 || D <= 0) return 0;
    // whatever the type and the alignment: the most planes of the forms that take rows of this
    // width (the two-pass form: row sums too, and the widest packs have the most row ranges)
    int64_t planes = M < kPlanSms ? M : kPlanSms;
    if (D <= kNarrowWidth && (narrow_workers(M, D) + 3) / 4 * 4 > planes) planes = (narrow_workers(M, D) + 3) / 4 * 4;
    size_t sums = 0;
    if (D * 4 > kMaxRowBytes) {
        sums = round256((size_t)M * sizeof(float2));
        if (wide_row_ranges(M, D, 8) > planes) planes = wide_row_ranges(M, D, 8);
    }
    return sums + 2 * round256((size_t)planes * D * 4);
}

swiglu_status swiglu_mlp_layer_norm_bwd(const void* dy, int64_t lddy, const void* s, int64_t lds, const void* gamma,
                                        const float* mean, const float* rstd, const void* dskip, int64_t ldskip,
                                        void* dx, int64_t lddx, void* dgamma, void* dbeta, int64_t M, int64_t D,
                                        int type, int param_type, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    swiglu_status rc = norm_check(M, D, type, param_type);
    if (rc != SWIGLU_OK) return rc;
    const size_t n = type_bytes(type), np = type_bytes(param_type);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int sms;
    if (misaligned(dgamma, np) || misaligned(dbeta, np))
        return fail(SWIGLU_ERR_MISALIGNED, "layer norm: a pointer is not aligned to its element");
    if (M == 0) {
        rc = device_sms(&sms);
        if (rc != SWIGLU_OK) return rc;
        for (void* p : {dgamma, dbeta}) {
            cudaError_t e = p ? cudaMemsetAsync(p, 0, (size_t)D * np, st) : cudaSuccess;
            if (e != cudaSuccess) return fail(SWIGLU_ERR_CUDA, "cudaMemsetAsync(parameter gradients)", e);
        }
        return SWIGLU_OK;
    }
    if (!dy || !s || !mean || !rstd || !dx || !workspace)
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a required pointer is null");
    if (lddy < D || lds < D || lddx < D || (dskip && ldskip < D))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a row stride is smaller than the width");
    if (misaligned(dy, n) || misaligned(s, n) || misaligned(dskip, n) || misaligned(dx, n) || misaligned(gamma, np) ||
        misaligned(mean, 4) || misaligned(rstd, 4) || !aligned16(workspace))
        return fail(SWIGLU_ERR_MISALIGNED, "layer norm: a pointer is not aligned to its element, or the workspace to 16 bytes");
    if (workspace_bytes < swiglu_mlp_layer_norm_bwd_workspace_size(M, D))
        return fail(SWIGLU_ERR_WORKSPACE_TOO_SMALL, "layer norm: workspace smaller than the size query returns");
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    Aligned v{(int)n};
    v.add(dy, lddy), v.add(s, lds), v.add(dskip, ldskip), v.add(dx, lddx), v.add(dy, D);
    if (D * (int64_t)n > kMaxRowBytes) v.add(gamma, 0);   // read in packs there
    const NormPlan p = bwd_plan(M, D, (int)n, dskip != nullptr);
    const bool shift = !v.ok(), wide = shift ? D > kNarrowWidth : D * (int64_t)n > kMaxRowBytes;
    // a worker of one warp comes with three others
    const int planes = (int)(wide    ? wide_row_ranges(M, D, shift ? 1 : 16 / (int)n)
                             : shift ? narrow_threads(D) == 32 ? (narrow_workers(M, D) + 3) / 4 * 4 : narrow_workers(M, D)
                                     : bwd_ctas(M, p));
    uint8_t* w = static_cast<uint8_t*>(workspace);
    float2* sums = reinterpret_cast<float2*>(w);
    if (wide) w += round256((size_t)M * sizeof(float2));
    float* pg = reinterpret_cast<float*>(w);
    float* pb = reinterpret_cast<float*>(w + round256((size_t)planes * D * 4));
    const NormBwd a{dy, s, gamma, dskip, mean, rstd, dx, dgamma ? pg : nullptr, dbeta ? pb : nullptr,
                    lddy, lds, ldskip, lddx, M, (int)D, p.lanes, param_type == SWIGLU_FP32};
    rc = launch_traced(SWIGLU_KERNEL_NORM_BWD, st,
                       [&] { return with_type(type, LaunchBwd{a, p, shift, sums, planes, st}); });
    if (rc != SWIGLU_OK || (!dgamma && !dbeta)) return rc;
    return launch_traced(SWIGLU_KERNEL_NORM_PARAMS, st, [&] {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)((D + 31) / 32), 2);
        cfg.blockDim = dim3(32, 16);
        cfg.stream = st;
        const float *g = pg, *b = pb;
        const int d = (int)D;
        if (param_type == SWIGLU_FP32)
            return cudaLaunchKernelEx(&cfg, layer_norm_params_kernel<float>, g, b, (float*)dgamma, (float*)dbeta, planes, d);
        if (param_type == SWIGLU_FP16)
            return cudaLaunchKernelEx(&cfg, layer_norm_params_kernel<__half>, g, b, (__half*)dgamma, (__half*)dbeta, planes, d);
        return cudaLaunchKernelEx(&cfg, layer_norm_params_kernel<__nv_bfloat16>, g, b, (__nv_bfloat16*)dgamma,
                                  (__nv_bfloat16*)dbeta, planes, d);
    });
}

}  // extern "C"
