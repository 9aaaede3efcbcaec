// layer_norm.cu -- layer norm forward and backward (include/swiglu_ops.h).
//
// Both directions are bound by HBM: a row is read once into registers, its statistics are
// reduced there, and the result is written once.  A row belongs to `lanes` threads, each
// holding CPT of its columns as packs of VEC elements (pack i of lane l is columns
// (i * lanes + l) * VEC ...), and a CTA walks rows blockIdx, blockIdx + gridDim, ...,
// loading its next row before it reduces the current one, so that loads stay in flight
// through the reductions.
#include "../host.h"
#include "convert.cuh"
#include "swiglu_ops.h"

namespace swiglu {
namespace {

constexpr int kPlanSms = 152;      // grids are planned for the GB300, so that the workspace query sees no device
constexpr int kMaxThreads = 1024;
constexpr int kMaxWidthFwd = 16384;   // widest rows held in registers: 1024 threads x 16 columns forward,
constexpr int kMaxWidthBwd = 8192;    // 8 backward, whose threads also hold two column sums for each column

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

// gamma or beta at column `col`, in the row's type or in fp32.
template <class T, int VEC>
__device__ __forceinline__ void load_param(float* o, const void* p, int gf32, int col, float none) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = none;
    } else if (gf32) {
        constexpr int V4 = VEC >= 4 ? 4 : 1;
#pragma unroll
        for (int q = 0; q < VEC / V4; ++q) {
            const Pack<float, V4> w = load_pack<float, V4>(static_cast<const float*>(p) + col + q * V4);
#pragma unroll
            for (int j = 0; j < V4; ++j) o[q * V4 + j] = w.v[j];
        }
    } else {
        const Pack<T, VEC> w = load_pack<T, VEC>(static_cast<const T*>(p) + col);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = to_f32(w.v[j]);
    }
}

// Sums over the `lanes` threads of a row.  One warp: shuffles.  The whole CTA: shuffles,
// then every thread adds the warps' sums from shared memory in warp order.  The caller
// alternates `buf`, so one barrier per reduction is enough: a buffer is rewritten only
// after the other one's barrier, which every reader of the first has passed.
constexpr int kWarps = kMaxThreads / 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float row_sum(float v, int lanes, float (*red)[kWarps], int buf) {
    v = warp_sum(v);
    if (lanes == 32) return v;
    if ((threadIdx.x & 31) == 0) red[buf][threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w += 4) {
        if (w * 32 < lanes) {
            const float4 q = *reinterpret_cast<const float4*>(&red[buf][w]);
            t += (q.x + q.y) + (q.z + q.w);
        }
    }
    return t;
}

__device__ __forceinline__ float2 row_sum2(float2 v, int lanes, float2 (*red)[kWarps], int buf) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (lanes == 32) return v;
    if ((threadIdx.x & 31) == 0) red[buf][threadIdx.x >> 5] = v;
    __syncthreads();
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; w += 2) {
        if (w * 32 < lanes) {
            const float4 q = *reinterpret_cast<const float4*>(&red[buf][w]);
            t.x += q.x + q.z;
            t.y += q.y + q.w;
        }
    }
    return t;
}

template <class T, int VEC, int CPT>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_fwd_kernel(const NormFwd a) {
    constexpr int NV = CPT / VEC;
    __shared__ __align__(16) float red[2][kWarps];
    const int lanes = a.lanes, lane = threadIdx.x % lanes, hop = lanes * VEC;
    const int rows = blockDim.x / lanes;                   // 1 unless a row is one warp
    if (threadIdx.x < 2 * kWarps) red[0][threadIdx.x] = 0.f;
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t row = (int64_t)blockIdx.x * rows + threadIdx.x / lanes;
    const int col = lane * VEC;                            // columns col + q * hop + j
    const T* x = static_cast<const T*>(a.x) + col;
    const T* r = static_cast<const T*>(a.r) + col;
    Pack<T, VEC> px[NV], pr[NV];
    auto load_row = [&](int64_t i) {
        const T* xi = x + i * a.ldx;
        const T* ri = r + i * a.ldr;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            if (col + q * hop < a.D) {
                px[q] = load_pack<T, VEC>(xi + q * hop);
                if (a.r) pr[q] = load_pack<T, VEC>(ri + q * hop);
            }
        }
    };
    if (row < a.M) load_row(row);
    const float inv = 1.f / (float)a.D;
    for (; row < a.M; row += step) {
        float v[CPT];
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float f = 0.f;
                if (col + q * hop < a.D) {
                    f = to_f32(px[q].v[j]);
                    if (a.r) f += to_f32(pr[q].v[j]);
                }
                v[q * VEC + j] = f;
                sum += f;
            }
        }
        if (row + step < a.M) load_row(row + step);
        if (a.r) {
            T* si = static_cast<T*>(a.s) + row * a.lds + col;
#pragma unroll
            for (int q = 0; q < NV; ++q)
                if (col + q * hop < a.D) store_pack<T, VEC>(si + q * hop, v + q * VEC);
        }
        const float mean = row_sum(sum, lanes, red, 0) * inv;
        float sq = 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            if (col + q * hop < a.D) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float c = v[q * VEC + j] - mean;
                    v[q * VEC + j] = c;
                    sq += c * c;
                }
            }
        }
        const float var = row_sum(sq, lanes, red, 1) * inv;
        const float rstd = __frsqrt_rn(var + a.eps);
        T* yi = static_cast<T*>(a.y) + row * a.ldy + col;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            if (col + q * hop < a.D) {
                float g[VEC], b[VEC];
                load_param<T, VEC>(g, a.gamma, a.gf32, col + q * hop, 1.f);
                load_param<T, VEC>(b, a.beta, a.gf32, col + q * hop, 0.f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) g[j] = v[q * VEC + j] * rstd * g[j] + b[j];
                store_pack<T, VEC>(yi + q * hop, g);
            }
        }
        if (lane == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

// A row wider than the registers hold: three passes over it, the last two from L2.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_fwd_wide_kernel(const NormFwd a) {
    __shared__ __align__(16) float red[2][kWarps];
    if (threadIdx.x < 2 * kWarps) red[0][threadIdx.x] = 0.f;
    __syncthreads();
    const float inv = 1.f / (float)a.D;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* r = a.r ? static_cast<const T*>(a.r) + row * a.ldr : nullptr;
        auto load = [&](int col, float* v) {
            const Pack<T, VEC> p = load_pack<T, VEC>(x + col);
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = to_f32(p.v[j]);
            if (r) {
                const Pack<T, VEC> e = load_pack<T, VEC>(r + col);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] += to_f32(e.v[j]);
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
        const float mean = row_sum(sum, blockDim.x, red, 0) * inv;
        for (int64_t c = first; c < a.D; c += hop) {
            load((int)c, v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sq += (v[j] - mean) * (v[j] - mean);
        }
        const float rstd = __frsqrt_rn(row_sum(sq, blockDim.x, red, 1) * inv + a.eps);
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

// Backward: the row's two sums, dx, and fp32 column sums of dy * xh and dy over the CTA's
// rows, kept in registers and written once as this CTA's partial plane.  A row stays in
// registers as it was loaded; xh and g are computed from it twice, before and after the
// reduction, which costs less than keeping them beside the column sums.
template <class T, int VEC, int CPT>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_bwd_kernel(const NormBwd a) {
    constexpr int NV = CPT / VEC;
    __shared__ __align__(16) float2 red[2][kWarps];
    extern __shared__ float acc[];                         // rows > 1: [2][D] sums of the CTA's warps
    const int lanes = a.lanes, lane = threadIdx.x % lanes, group = threadIdx.x / lanes, hop = lanes * VEC;
    const int rows = blockDim.x / lanes;
    if (threadIdx.x < 2 * kWarps) red[0][threadIdx.x] = make_float2(0.f, 0.f);
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t row = (int64_t)blockIdx.x * rows + group;
    const int col = lane * VEC;                            // columns col + q * hop + j
    const T* dy = static_cast<const T*>(a.dy) + col;
    const T* s = static_cast<const T*>(a.s) + col;
    Pack<T, VEC> py[NV], ps[NV];
    float mean = 0.f, rstd = 0.f;
    auto load_row = [&](int64_t i) {
        mean = a.mean[i];
        rstd = a.rstd[i];
        const T* yi = dy + i * a.lddy;
        const T* si = s + i * a.lds;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            if (col + q * hop < a.D) {
                py[q] = load_pack<T, VEC>(yi + q * hop);
                ps[q] = load_pack<T, VEC>(si + q * hop);
            }
        }
    };
    float dg[CPT], db[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) dg[j] = db[j] = 0.f;
    if (row < a.M) load_row(row);
    const float inv = 1.f / (float)a.D;
    int buf = 0;
    for (; row < a.M; row += step, buf ^= 1) {
        Pack<T, VEC> cy[NV], cs[NV], pk[NV];
        const float mu = mean, rs = rstd;
#pragma unroll
        for (int q = 0; q < NV; ++q) cy[q] = py[q], cs[q] = ps[q];
        if (a.skip) {
            const T* ki = static_cast<const T*>(a.skip) + row * a.ldk + col;
#pragma unroll
            for (int q = 0; q < NV; ++q)
                if (col + q * hop < a.D) pk[q] = load_pack<T, VEC>(ki + q * hop);
        }
        if (row + step < a.M) load_row(row + step);
        float2 c = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            if (col + q * hop < a.D) {
                float w[VEC];
                load_param<T, VEC>(w, a.gamma, a.gf32, col + q * hop, 1.f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float d = to_f32(cy[q].v[j]), xh = (to_f32(cs[q].v[j]) - mu) * rs, g = d * w[j];
                    dg[q * VEC + j] += d * xh;
                    db[q * VEC + j] += d;
                    c.x += g;
                    c.y += g * xh;
                }
            }
        }
        c = row_sum2(c, lanes, red, buf);
        c.x *= inv;
        c.y *= inv;
        T* oi = static_cast<T*>(a.dx) + row * a.lddx + col;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            if (col + q * hop < a.D) {
                float w[VEC];
                load_param<T, VEC>(w, a.gamma, a.gf32, col + q * hop, 1.f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float xh = (to_f32(cs[q].v[j]) - mu) * rs;
                    w[j] = rs * (to_f32(cy[q].v[j]) * w[j] - c.x - xh * c.y);
                    if (a.skip) w[j] += to_f32(pk[q].v[j]);
                }
                store_pack<T, VEC>(oi + q * hop, w);
            }
        }
    }
    if (a.pg == nullptr && a.pb == nullptr) return;
    if (rows > 1) {
        // one warp per row: add the warps' sums in warp order, through shared memory
        for (int w = 0; w < rows; ++w) {
            if (group == w) {
#pragma unroll
                for (int k = 0; k < CPT; ++k) {
                    const int at = col + k / VEC * hop + k % VEC;
                    if (at < a.D) {
                        if (w > 0) {
                            dg[k] += acc[at];
                            db[k] += acc[a.D + at];
                        }
                        acc[at] = dg[k];
                        acc[a.D + at] = db[k];
                    }
                }
            }
            __syncthreads();
        }
        if (group != rows - 1) return;
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int at = col + k / VEC * hop + k % VEC;
        if (at < a.D) {
            if (a.pg) a.pg[(int64_t)blockIdx.x * a.D + at] = dg[k];
            if (a.pb) a.pb[(int64_t)blockIdx.x * a.D + at] = db[k];
        }
    }
}

// Rows wider than the registers hold, in two passes: the two sums of every row, then dx
// and the column sums of a block of columns over a range of rows.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_bwd_wide_sums_kernel(const NormBwd a, float2* sums) {
    __shared__ __align__(16) float2 red[2][kWarps];
    if (threadIdx.x < 2 * kWarps) red[0][threadIdx.x] = make_float2(0.f, 0.f);
    __syncthreads();
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, buf ^= 1) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const T* s = static_cast<const T*>(a.s) + row * a.lds;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float2 c = make_float2(0.f, 0.f);
        for (int64_t col = threadIdx.x * VEC; col < a.D; col += blockDim.x * VEC) {
            float w[VEC];
            const Pack<T, VEC> py = load_pack<T, VEC>(dy + col), ps = load_pack<T, VEC>(s + col);
            load_param<T, VEC>(w, a.gamma, a.gf32, (int)col, 1.f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = to_f32(py.v[j]) * w[j];
                c.x += g;
                c.y += g * ((to_f32(ps.v[j]) - mean) * rstd);
            }
        }
        c = row_sum2(c, blockDim.x, red, buf);
        if (threadIdx.x == 0) sums[row] = make_float2(c.x / (float)a.D, c.y / (float)a.D);
    }
}

// grid (column blocks, row ranges): CTA (x, y) has columns x * blockDim * VEC ... and rows
// y, y + gridDim.y, ...; its column sums are partial plane y.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_bwd_wide_kernel(const NormBwd a, const float2* sums) {
    const int64_t col = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (col >= a.D) return;
    float w[VEC], dg[VEC], db[VEC];
    load_param<T, VEC>(w, a.gamma, a.gf32, (int)col, 1.f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[j] = db[j] = 0.f;
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
        const Pack<T, VEC> py = load_pack<T, VEC>(static_cast<const T*>(a.dy) + row * a.lddy + col);
        const Pack<T, VEC> ps = load_pack<T, VEC>(static_cast<const T*>(a.s) + row * a.lds + col);
        const float mean = a.mean[row], rstd = a.rstd[row];
        const float2 c = sums[row];
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = to_f32(py.v[j]), xh = (to_f32(ps.v[j]) - mean) * rstd;
            dg[j] += d * xh;
            db[j] += d;
            o[j] = rstd * (d * w[j] - c.x - xh * c.y);
        }
        if (a.skip) {
            const Pack<T, VEC> pk = load_pack<T, VEC>(static_cast<const T*>(a.skip) + row * a.ldk + col);
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] += to_f32(pk.v[j]);
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
    if (col < D) {
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

// How a launch covers its rows.  Up to 256 columns a row is one warp (no barriers) and a
// CTA holds four rows; wider rows get one CTA with 8 columns a thread, 16 above 8192.
struct NormPlan {
    int cpt, lanes, threads;
    int rows() const { return threads / lanes; }
};

NormPlan norm_plan(int64_t D) {
    NormPlan p;
    p.cpt = D <= 8192 ? 8 : 16;
    p.lanes = (int)(D > kMaxWidthFwd ? kMaxThreads : ((D + p.cpt - 1) / p.cpt + 31) / 32 * 32);
    p.threads = p.lanes == 32 ? 128 : p.lanes;
    return p;
}

// CTAs of the backward = partial planes.  About 1024 threads an SM keep two rows of loads in flight.
int64_t bwd_ctas(int64_t M, const NormPlan& p) {
    const int64_t want = (M + p.rows() - 1) / p.rows();
    const int64_t most = (int64_t)kPlanSms * (1024 / p.threads < 8 ? 1024 / p.threads : 8);
    return want < most ? want : most;
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

// Elements moved at a time: 16 bytes where every base, row stride and the width allow it,
// 4 bytes (two 16-bit elements) where those are even, else one.
struct Vec {
    int size, bits = 0;
    void add(const void* p, int64_t ld) {
        if (p) bits |= (int)(reinterpret_cast<uintptr_t>(p) & 15) | (int)((ld * size) & 15);
    }
    int elements() const { return (bits & 15) == 0 ? 16 / size : size == 2 && (bits & 3) == 0 ? 2 : 1; }
};

// f.run<T, VEC>() for the run-time type and pack width.
template <class F>
cudaError_t with_types(int type, int vec, const F& f) {
    if (type == SWIGLU_FP32) return vec == 4 ? f.template run<float, 4>() : f.template run<float, 1>();
    if (type == SWIGLU_FP16)
        return vec == 8 ? f.template run<__half, 8>() : vec == 2 ? f.template run<__half, 2>() : f.template run<__half, 1>();
    return vec == 8   ? f.template run<__nv_bfloat16, 8>()
           : vec == 2 ? f.template run<__nv_bfloat16, 2>()
                      : f.template run<__nv_bfloat16, 1>();
}

struct LaunchFwd {
    const NormFwd& a;
    const NormPlan& p;
    cudaStream_t s;
    template <class T, int VEC>
    cudaError_t run() const {
        const int64_t want = (a.M + p.rows() - 1) / p.rows();
        const int64_t most = (int64_t)kPlanSms * (2048 / p.threads < 16 ? 2048 / p.threads : 16);
        const unsigned grid = (unsigned)(want < most ? want : most);
        if (a.D > kMaxWidthFwd)
            layer_norm_fwd_wide_kernel<T, VEC><<<grid, kMaxThreads, 0, s>>>(a);
        else if (p.cpt == 16)
            layer_norm_fwd_kernel<T, VEC, 16><<<grid, p.threads, 0, s>>>(a);
        else
            layer_norm_fwd_kernel<T, VEC, 8><<<grid, p.threads, 0, s>>>(a);
        return cudaGetLastError();
    }
};

struct LaunchBwd {
    const NormBwd& a;
    const NormPlan& p;
    float2* sums;
    int planes;
    cudaStream_t s;
    template <class T, int VEC>
    cudaError_t run() const {
        if (a.D > kMaxWidthBwd) {
            const int64_t grid = a.M < kPlanSms * 2 ? a.M : kPlanSms * 2;
            layer_norm_bwd_wide_sums_kernel<T, VEC><<<(unsigned)grid, kMaxThreads, 0, s>>>(a, sums);
            const dim3 tiles((unsigned)((a.D + 256 * VEC - 1) / (256 * VEC)), (unsigned)planes);
            layer_norm_bwd_wide_kernel<T, VEC><<<tiles, 256, 0, s>>>(a, sums);
        } else {
            const size_t smem = p.rows() > 1 ? 2 * (size_t)a.D * sizeof(float) : 0;
            layer_norm_bwd_kernel<T, VEC, 8><<<(unsigned)planes, p.threads, smem, s>>>(a);
        }
        return cudaGetLastError();
    }
};

swiglu_status norm_check(int64_t M, int64_t D, int type, int param_type) {
    if (M < 0 || D <= 0) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a size is negative or zero");
    if (M >= (int64_t(1) << 31) || D >= (int64_t(1) << 30))
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "layer norm: M must stay below 2^31 and D below 2^30");
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
    Vec v{(int)n};
    v.add(x, ldx), v.add(residual, ldr), v.add(y, ldy), v.add(s, lds), v.add(x, D);
    v.add(gamma, 0), v.add(beta, 0);
    const NormFwd a{x, residual, gamma, beta, y, s, mean, rstd, ldx, ldr, ldy, lds, M, (int)D, norm_plan(D).lanes,
                    param_type == SWIGLU_FP32, eps};
    const NormPlan p = norm_plan(D);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_NORM_FWD, st,
                         [&] { return with_types(type, v.elements(), LaunchFwd{a, p, st}); });
}

size_t swiglu_mlp_layer_norm_bwd_workspace_size(int64_t M, int64_t D) {
    if (M <= 0 || D <= 0) return 0;
    if (D > kMaxWidthBwd)   // row sums, then the planes of the narrowest packs (the most row ranges of any vec)
        return round256((size_t)M * sizeof(float2)) + 2 * round256((size_t)wide_row_ranges(M, D, 8) * D * 4);
    return 2 * round256((size_t)bwd_ctas(M, norm_plan(D)) * D * 4);
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
    Vec v{(int)n};
    v.add(dy, lddy), v.add(s, lds), v.add(dskip, ldskip), v.add(dx, lddx), v.add(dy, D), v.add(gamma, 0);
    const NormPlan p = norm_plan(D);
    const bool wide = D > kMaxWidthBwd;
    const int vec = v.elements();
    const int planes = (int)(wide ? wide_row_ranges(M, D, vec) : bwd_ctas(M, p));
    uint8_t* w = static_cast<uint8_t*>(workspace);
    float2* sums = reinterpret_cast<float2*>(w);
    if (wide) w += round256((size_t)M * sizeof(float2));
    float* pg = reinterpret_cast<float*>(w);
    float* pb = reinterpret_cast<float*>(w + round256((size_t)planes * D * 4));
    const NormBwd a{dy, s, gamma, dskip, mean, rstd, dx, dgamma ? pg : nullptr, dbeta ? pb : nullptr,
                    lddy, lds, ldskip, lddx, M, (int)D, p.lanes, param_type == SWIGLU_FP32};
    rc = launch_traced(SWIGLU_KERNEL_NORM_BWD, st,
                       [&] { return with_types(type, vec, LaunchBwd{a, p, sums, planes, st}); });
    if (rc != SWIGLU_OK || (!dgamma && !dbeta)) return rc;
    return launch_traced(SWIGLU_KERNEL_NORM_PARAMS, st, [&] {
        const dim3 grid((unsigned)((D + 31) / 32), 2), block(32, 16);
        if (param_type == SWIGLU_FP32)
            layer_norm_params_kernel<float><<<grid, block, 0, st>>>(pg, pb, (float*)dgamma, (float*)dbeta, planes, (int)D);
        else if (param_type == SWIGLU_FP16)
            layer_norm_params_kernel<__half><<<grid, block, 0, st>>>(pg, pb, (__half*)dgamma, (__half*)dbeta, planes, (int)D);
        else
            layer_norm_params_kernel<__nv_bfloat16>
                <<<grid, block, 0, st>>>(pg, pb, (__nv_bfloat16*)dgamma, (__nv_bfloat16*)dbeta, planes, (int)D);
        return cudaGetLastError();
    });
}

}  // extern "C"
