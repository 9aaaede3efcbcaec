// layer_norm_fwd.cu -- layer norm forward (include/swiglu_ops.h).
//
// Bound by HBM: a row is read once into registers, its statistics are reduced there, and the
// result is written once.  At the HBM rate an SM has about 40 instructions a column for all of
// it, so what a row costs besides its columns has to be spread over many of them, and the
// columns' arithmetic runs in packed pairs: a row belongs to a group of `lanes` threads with NV
// packs of 16 bytes each (pack k = q * lanes + lane of the row, q < NV).  Measured, 11136 x 3584
// bf16 with the residual stream's sum, 319 MB: 53.6 us, 6.0 TB/s of the 6.78 TB/s of a copy.
#include <algorithm>

#include "layer_norm.cuh"

namespace swiglu {
namespace {

struct NormFwd {
    const void *x, *r, *gamma, *beta;
    void *y, *s;
    float *mean, *rstd;
    int64_t ldx, ldr, ldy, lds, M;
    int D, lanes, gf32;
    float eps;
};

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

// ---------------------------------------------------------------- forward

// One row for each group of `lanes` threads: a CTA is one row of more than a warp, or four
// rows of one.  Many small CTAs take turns at loading, reducing and storing; a persistent
// form with the next row in flight in shared memory took 57 us where this takes 53
// (11136 x 3584 bf16).  The statistics need one barrier: a warp centres its columns on its
// own mean, and the warps' (mean, sum of squares about it) are joined exactly.  EDGE: rows off
// 16-byte boundaries, all tensors alike; as many CTAs as the SMs hold walk the rows, a multiple of
// 152 rows, that is of whole packs, apart, so that gamma and beta go to shared memory once a CTA
// (once a row, 11136 x 3583 bf16 took 187 us).
template <class T, int NV, bool RES, bool EDGE, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) layer_norm_fwd_kernel(const NormFwd a) {
    constexpr int V = kVec<T>, P = V / 2;
    __shared__ float2 both[EDGE ? 2 : 1][THREADS / 32];
    extern __shared__ uint4 smem[];        // EDGE: gamma and beta of every row of the CTA, fp32, in packs
    const int lanes = a.lanes, lane = threadIdx.x % lanes, D = a.D;
    int64_t row = (int64_t)blockIdx.x * (blockDim.x / lanes) + threadIdx.x / lanes;
    if (row >= a.M) return;                // whole warps; with more than one warp a row, no thread
    const int m = EDGE ? into_pack<T>(a.x, row, a.ldx) : 0, end = D + m, width = padded(D + V - 1);
    if (EDGE) {
        float* g = reinterpret_cast<float*>(smem) + threadIdx.x / lanes * 2 * width;
        stage_param<T>(g, a.gamma, a.gf32, D, m, width, 1.f, lane, lanes);
        stage_param<T>(g + width, a.beta, a.gf32, D, m, width, 0.f, lane, lanes);
        if (lanes == 32) __syncwarp();
        else __syncthreads();
    }
    const uint32_t params = EDGE ? (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x / lanes * 2 * width * 4 : 0;
    int buf = 0;
    do {
        float2* red = both[buf];
        const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row * a.ldx - m);
        const uint4* r = reinterpret_cast<const uint4*>(static_cast<const T*>(a.r) + row * a.ldr - m);
        const bool inside = row > 0 && row < a.M - 1;      // the first and the last pack are the tensors', too
        F2 v[NV * P];
        {
            uint4 px[NV], pr[NV];
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int k = q * lanes + lane;
                px[q] = pr[q] = make_uint4(0, 0, 0, 0);
                if (EDGE && !inside && on_edge<T, NV>(q, k, m, end)) {
                    px[q] = load_edge<T>(reinterpret_cast<const T*>(x) + m, k * V - m, D);
                    if (RES) pr[q] = load_edge<T>(reinterpret_cast<const T*>(r) + m, k * V - m, D);
                } else if (in_row<T, NV>(q, k, end)) {
                    px[q] = __ldcs(x + k);
                    if (RES) pr[q] = __ldcs(r + k);
                }
            }
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                F2* w = v + q * P;
                const int k = q * lanes + lane;
                if (EDGE && on_edge<T, NV>(q, k, m, end)) {
                    px[q] = row_elements<T>(px[q], k * V - m, D);
                    if (RES) pr[q] = row_elements<T>(pr[q], k * V - m, D);
                }
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
            T* s = static_cast<T*>(a.s) + row * a.lds - m;
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int k = q * lanes + lane;
                if (EDGE && on_edge<T, NV>(q, k, m, end)) store_edge<T>(s + m, k * V - m, D, pack16<T>(v + q * P));
                else if (in_row<T, NV>(q, k, end)) reinterpret_cast<uint4*>(s)[k] = pack16<T>(v + q * P);
            }
        }
        F2 sum2 = f2(0.f);
#pragma unroll
        for (int i = 0; i < NV * P; ++i) sum2 = sum2 + v[i];
        // columns of warp w: of every pack its 32 * V from (q * lanes + 32 w) * V
        auto columns = [&](int w) {
            int n = w == 0 ? -m : 0;
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int left = end - (q * lanes + 32 * w) * V;
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
            const int k = q * lanes + lane;
            if (EDGE && on_edge<T, NV>(q, k, m, end)) {        // the elements that are not the row's add nothing
                float e[V];
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 c = split(v[q * P + i] + mu);
                    e[2 * i] = c.x, e[2 * i + 1] = c.y;
                }
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if ((unsigned)(k * V - m + j) >= (unsigned)D) e[j] = 0.f;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const F2 c = f2(e[2 * i], e[2 * i + 1]);
                    sq2 = fma(c, c, sq2);
                }
            } else if (in_row<T, NV>(q, k, end)) {
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
            const int w = threadIdx.x & 31;    // lane w of every warp takes warp w's
            const float2 part = w < warps ? red[w] : make_float2(0.f, 0.f);
            const float n = w < warps ? columns(w) : 0.f;
            mean = warp_sum(n * part.x) / (float)D;
            const float d = part.x - mean;
            sq = warp_sum(part.y + n * d * d);
        }
        const float rstd = __frsqrt_rn(sq / (float)D + a.eps);
        const F2 rs = f2(rstd), m2 = f2(-mean);
        T* y = static_cast<T*>(a.y) + row * a.ldy - m;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane;
            if (in_row<T, NV>(q, k, end)) {
                F2 g[P], b[P];
                if constexpr (EDGE) {
                    load_staged<T>(g, params, k, width);
                    load_staged<T>(b, params + width * 4, k, width);
                } else {
                    load_param16<T>(g, a.gamma, a.gf32, k, 1.f);
                    load_param16<T>(b, a.beta, a.gf32, k, 0.f);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) g[i] = fma((v[q * P + i] + m2) * rs, g[i], b[i]);
                if (EDGE && on_edge<T, NV>(q, k, m, end)) store_edge<T>(y + m, k * V - m, D, pack16<T>(g));
                else __stcs(reinterpret_cast<uint4*>(y) + k, pack16<T>(g));
            }
        }
        if (lane == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        row += (int64_t)gridDim.x * (blockDim.x / lanes);
        if (EDGE) buf ^= 1;                // a buffer is written again after the next row's barrier
    } while (EDGE && row < a.M);
}

// Bound by instructions: 4099 x 1021 fp32 9.3 us, 3.6 TB/s (with twice the columns a thread, half of them
// past the row, 11.5); 40000 x 257 bf16 22.3 us, 1.8 TB/s.
template <class T, bool RES, int THREADS, int COLS>
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
    float v[COLS];
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
        v[i] = 0.f;
        if (t + i * THREADS < D) v[i] = to_f32(x[i * THREADS]);
    }
    if (RES) {
        T* s = static_cast<T*>(a.s) + row * a.lds + t;
#pragma unroll
        for (int i = 0; i < COLS; ++i)
            if (t + i * THREADS < D) v[i] += to_f32(r[i * THREADS]);
#pragma unroll
        for (int i = 0; i < COLS; ++i)
            if (t + i * THREADS < D) s[i * THREADS] = from_f32<T>(v[i]);
    }
    float sum = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < COLS; ++i) sum += v[i];
    const float mean = row_sum(sum, 0, THREADS, red, 0) / (float)D;
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
        v[i] -= mean;
        if (t + i * THREADS < D) sq += v[i] * v[i];
    }
    const float rstd = __frsqrt_rn(row_sum(sq, 0, THREADS, red, 1) / (float)D + a.eps);
    T* y = static_cast<T*>(a.y) + row * a.ldy + t;
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
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

// A row wider than the registers hold: three passes over it, the last two mostly from L2 (16-byte
// packs where rows and parameters allow them; 3000 x 14001 bf16, which single elements took 146
// us for, took 68 in shifted packs, so these are rows past 64 KB, or apart).  Measured with the
// residual stream's sum: 3000 x 40000 bf16, 960 MB, 226 us, 4.2 TB/s; single elements, bound by
// instructions, 3000 x 40001: 543 us (with runs unrolled by 1 instead of 2 716, by 4 781).
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
        float v[VEC];
        LongSum sum, sq;
        constexpr int run = VEC > 1 ? 1 : kRun;
        for (int64_t c = first; c < a.D;) {
            float part = 0.f;
#pragma unroll 2
            for (int i = 0; i < run && c < a.D; ++i, c += hop) {
                load((int)c, v);
#pragma unroll
                for (int j = 0; j < VEC; ++j) part += v[j];
            }
            sum.add(part);
        }
        const float mean = row_sum(sum.value(), 0, blockDim.x, red, 0) * inv;
        for (int64_t c = first; c < a.D;) {
            float part = 0.f;
#pragma unroll 2
            for (int i = 0; i < run && c < a.D; ++i, c += hop) {
                load((int)c, v);
#pragma unroll
                for (int j = 0; j < VEC; ++j) part += (v[j] - mean) * (v[j] - mean);
            }
            sq.add(part);
        }
        const float rstd = __frsqrt_rn(row_sum(sq.value(), 0, blockDim.x, red, 1) * inv + a.eps);
        for (int64_t c = first; c < a.D; c += hop) {
            float g[VEC], b[VEC];
            load((int)c, v);
            // not before the last pass over x and the residual, in whose place s may be
            if (r) store_pack<T, VEC>(static_cast<T*>(a.s) + row * a.lds + c, v);
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

// ---------------------------------------------------------------- host side

// Packs a thread holds at most, and the widest row of 1024 threads' packs: 64 KB.
constexpr int kFwdPacks = 4;
constexpr int64_t kFwdRowBytes = 1024 * kFwdPacks * 16;

// Forward: CTAs of one row of more than a warp, or of four rows of one.
NormPlan fwd_plan(int64_t width, int size) {
    NormPlan p = norm_plan(width, size, kFwdPacks, 128);
    if (p.lanes > 32) p.groups = 1;
    return p;
}

struct LaunchFwd {
    const NormFwd& a;
    const NormPlan& p;
    Lie lie;
    cudaStream_t s;
    template <class T, int NV, bool RES, bool EDGE>
    cudaError_t go() const {
        // 64 registers for the small CTAs, whose number hides the latencies; the larger ones
        // all hold 4 packs a thread
        auto kern = layer_norm_fwd_kernel<T, NV, RES, EDGE, 128, EDGE ? 6 : 8>;
        if constexpr (NV == 4) {
            if (p.threads() > 384) kern = layer_norm_fwd_kernel<T, NV, RES, EDGE, 1024, 1>;
            else if (p.threads() > 128) kern = layer_norm_fwd_kernel<T, NV, RES, EDGE, 384, 2>;
        }
        const size_t smem = EDGE ? (size_t)p.groups * 2 * padded((int)reach(a.D, (int)sizeof(T), true)) * 4 : 0;
        cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
        int64_t grid = (a.M + p.groups - 1) / p.groups;
        if (EDGE) {
            const int64_t by_threads = p.threads() > 384 ? 1 : p.threads() > 128 ? 2 : 6, by_smem = (int64_t)(kSmem / (smem + 2048));
            grid = std::min(grid, kPlanSms * std::max<int64_t>(1, std::min(by_threads, by_smem)));
        }
        kern<<<(unsigned)grid, p.threads(), smem, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int NV>
    cudaError_t res() const {
        if (lie == kEdge) return a.r ? go<T, NV, true, true>() : go<T, NV, false, true>();
        return a.r ? go<T, NV, true, false>() : go<T, NV, false, false>();
    }
    template <class T, int THREADS, int COLS>
    cudaError_t narrow() const {
        constexpr int rows = THREADS == 32 ? 4 : 1;
        auto kern = a.r ? layer_norm_fwd_narrow_kernel<T, true, THREADS, COLS> : layer_norm_fwd_narrow_kernel<T, false, THREADS, COLS>;
        kern<<<(unsigned)((a.M + rows - 1) / rows), THREADS * rows, 0, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int THREADS>
    cudaError_t narrow() const {           // half as many columns a thread where they are enough
        return a.D <= THREADS * kCols / 2 ? narrow<T, THREADS, kCols / 2>() : narrow<T, THREADS, kCols>();
    }
    template <class T>
    cudaError_t run() const {
        if (lie == kApart ? a.D > kNarrowWidth : (int64_t)a.D * (int)sizeof(T) > kFwdRowBytes) {
            const unsigned grid = (unsigned)(a.M < kPlanSms * 4 ? a.M : kPlanSms * 4);
            if (lie == kApart) layer_norm_fwd_wide_kernel<T, 1><<<grid, kMaxThreads, 0, s>>>(a);
            else layer_norm_fwd_wide_kernel<T, kVec<T>><<<grid, kMaxThreads, 0, s>>>(a);
            return cudaGetLastError();
        }
        if (lie == kApart) {
            const int n = narrow_threads(a.D);
            return n == 32 ? narrow<T, 32>() : n == 128 ? narrow<T, 128>() : narrow<T, 512>();
        }
        return p.nv == 1 ? res<T, 1>() : p.nv == 2 ? res<T, 2>() : p.nv == 3 ? res<T, 3>() : res<T, 4>();
    }
};

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
    if (y == s) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: y and s are the same");
    if (ldx < D || ldy < D || (residual && (ldr < D || lds < D)))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a row stride is smaller than the width");
    const size_t n = type_bytes(type), np = type_bytes(param_type);
    if (misaligned(x, n) || misaligned(y, n) || misaligned(residual, n) || misaligned(s, n) || misaligned(gamma, np) ||
        misaligned(beta, np) || misaligned(mean, 4) || misaligned(rstd, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "layer norm: a pointer is not aligned to its element");
    int sms;
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    Rows16 v{(int)n};
    v.add(x, ldx), v.add(residual, ldr), v.add(y, ldy), v.add(s, lds);
    Lie lie = v.lie(D);
    // parameters off 16-byte boundaries go through shared memory as the shifted rows' do
    if (lie == kWhole && (misaligned(gamma, 16) || misaligned(beta, 16))) lie = kEdge;
    const int64_t most = reach(D, (int)n, true);
    // Shifted packs pay where 2-byte accesses cost much: 16-bit rows of more than a warp's (element
    // by element, then packs, us: 40000 x 515 70, 31; 11136 x 3583 105, 41; but 40000 x 257 22.2, 24.0;
    // fp32 4099 x 1021 10.2, 13.9; 3000 x 7001 44.5, 55.7), and where a row has too many elements
    // for single ones.  Widest: their registers, and the parameters' 227 KB.
    if (lie == kEdge && D <= (n == 4 ? kNarrowWidth : 32 * kCols)) lie = kApart;
    if (lie == kEdge && (most * (int64_t)n > kFwdRowBytes || 2 * (most + 7) * 4 > (int64_t)kSmem - 1024)) lie = kApart;
    const NormPlan p = fwd_plan(reach(D, (int)n, lie == kEdge), (int)n);
    const NormFwd a{x, residual, gamma, beta, y, s, mean, rstd, ldx, ldr, ldy, lds, M, (int)D, p.lanes,
                    param_type == SWIGLU_FP32, eps};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_NORM_FWD, st, [&] { return with_type(type, LaunchFwd{a, p, lie, st}); });
}

}  // extern "C"
