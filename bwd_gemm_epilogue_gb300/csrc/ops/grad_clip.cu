// grad_clip.cu -- global norm of many gradients and their clipping (include/swiglu_ops.h).
//
// Two launches: sums of squares (one fp64 sum per CTA), then the scaling, whose CTAs each
// add those sums in the same order, so every one of them holds the same norm and no CTA
// waits for another.  The tensors' table travels in the kernels' parameters (no copy, no
// allocation, fit for stream capture).  All tensors, in granules of kGranule bytes, are
// divided evenly over the CTAs; a CTA walks its share tensor by tensor, 32 KB at a time,
// and the scaling walks it backwards, so that what the norm read last is still in L2.
//
// Bound by HBM: gradients larger than L2 are read twice (the factor needs all of them first) and
// written once.  Measured, 616.6 M bf16: 574 us, 3.7 GB at 6.4 TB/s of the 6.78 TB/s of a copy.
// Few and small gradients: two launches and one sum of the norm, 8.5 us.
#include <algorithm>
#include <memory>
#include <new>

#include "../host.h"
#include "convert.cuh"
#include "swiglu_ops.h"

namespace swiglu {
namespace {

constexpr int kPlanSms = 152;
constexpr int kThreads = 512;
// CTAs = fp64 sums of one launch, 2 an SM: fewer sums to add and fewer first loads than with more (2, 3
// and 4 an SM, us: 616.6 M bf16 574, 577, 584; 48 mixed tensors of 19 M elements 25.6, 27.1, 28.6; 51 of
// up to 0.5 M each 13.9, 17.3, 19.7; but 3 tensors of 0.4 M in all 8.6, 8.4, 8.4, and the norm alone of
// the first 180, 174).
constexpr int kCtas = kPlanSms * 2;
constexpr int kMaxTensors = 768;             // per launch: 22 KB of parameters
constexpr int kFewTensors = 64;              // a second, 2 KB table for the usual few (shorter launches)
constexpr int64_t kGranule = 16384;
constexpr int kBlock = 4;                    // 16-byte packs a thread loads at a time

template <int N>
struct ClipTable {
    const void* in[N];
    void* out[N];
    int64_t count[N];
    uint32_t first[N + 1];                   // first granule of each tensor; entry n: their number
    uint8_t type[N];
    int n;
};

__host__ __device__ constexpr int64_t granule_elements(int type) { return kGranule / (type == SWIGLU_FP32 ? 4 : 2); }

// This CTA's share of the granules: [begin, end).
template <int N>
__device__ __forceinline__ uint2 share_of(const ClipTable<N>& c) {
    const uint64_t all = c.first[c.n];
    return make_uint2((uint32_t)(all * blockIdx.x / gridDim.x), (uint32_t)(all * (blockIdx.x + 1) / gridDim.x));
}

// The tensor that has granule g.
template <int N>
__device__ __forceinline__ int tensor_of(const ClipTable<N>& c, uint32_t g) {
    int lo = 0, hi = c.n;                    // first[lo] <= g < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (c.first[mid] <= g) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Of n elements at p, those before the first 16-byte boundary.
template <class T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
    const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int64_t)sizeof(T);
    return h < n ? h : n;
}

// Packs from + j * kThreads (j < kBlock) of q, zeros past `packs`.
template <class T>
__device__ __forceinline__ void load_block(uint4* b, const T* q, int from, int packs) {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
        const int i = from + j * kThreads;
        b[j] = i < packs ? reinterpret_cast<const uint4*>(q)[i] : make_uint4(0, 0, 0, 0);
    }
}

// Sum of the squares of a block's elements times `scale`, 16 to each of two sums.
template <class T, bool SCALED>
__device__ __forceinline__ float block_squares(const uint4* b, float scale) {
    constexpr int V = 16 / sizeof(T);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
        F2 v[V / 2];
        unpack16<T>(b[j], v);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 f = split(SCALED ? v[i] * f2(scale) : v[i]);
            s0 += f.x * f.x;
            s1 += f.y * f.y;
        }
    }
    return s0 + s1;
}

// It is taken in fp32 as the elements are, and once more of their scaled values where that overflowed
// (finite elements above 1.8e19 do) or came out below kLeastSquares (elements below 1e-18 can): fp32
// squares under 1.2e-38 are off by up to 2^-150 each, 32 of them by 2e-44, which is 2^-28 of that least
// sum.  Times 2^100 (2^-100) every element that such a block can have, down to 2^-149 (up to 2^128),
// has a square in the normal range or one that does not count beside the block's largest.
constexpr float kLeastSquares = 1e-35f;

template <class T>
__device__ __noinline__ double block_squares_scaled(const T* q, int from, int packs, bool up) {
    uint4 b[kBlock];
    load_block(b, q, from, packs);
    const float f = block_squares<T, true>(b, up ? 0x1p100f : 0x1p-100f);
    return (double)f * (up ? 0x1p-200 : 0x1p200);
}
// Whether a block has an element other than 0 and -0, which whole gradients can consist of.
template <class T>
__device__ __forceinline__ bool any_element(const uint4* b) {
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < kBlock; ++j) any |= b[j].x | b[j].y | b[j].z | b[j].w;
    return (any & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) != 0;
}
template <class T>
__device__ __forceinline__ double squares(const T* p, int64_t n) {
    constexpr int V = 16 / sizeof(T);
    double s = 0.0;
    const int64_t head = head_of(p, n);
    const int packs = (int)((n - head) / V);
    const int64_t tail = head + (int64_t)packs * V;
    if (threadIdx.x < head) {
        const double v = to_f32(p[threadIdx.x]);
        s = v * v;
    }
    if (tail + threadIdx.x < n) {
        const double v = to_f32(p[tail + threadIdx.x]);
        s += v * v;
    }
    const T* q = p + head;
    for (int i = threadIdx.x; i < packs; i += kBlock * kThreads) {
        uint4 b[kBlock];
        load_block(b, q, i, packs);
        const float f = block_squares<T, false>(b, 1.f);
        const bool small = f < kLeastSquares && any_element<T>(b);
        s += small || isinf(f) ? block_squares_scaled(q, i, packs, small) : (double)f;
    }
    return s;
}

// Sum over the CTA's threads, in a fixed order; valid in thread 0.
__device__ __forceinline__ double cta_sum(double v) {
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) v += part[w];
    }
    return v;
}

// Sum of g^2 over this CTA's share: fp32 products and sums of 64 bytes a thread, then fp64.  Bound by
// HBM (1.23 GB of bf16 in 203 us, 6.1 TB/s); what hides the latency is 32 warps an SM with 64 bytes a
// thread in flight (two such blocks a thread, at 24 warps: 698 us with the scaling where one took 561).
template <int N>
__global__ void __launch_bounds__(kThreads, kCtas / kPlanSms) grad_squares_kernel(const __grid_constant__ ClipTable<N> c, double* sums) {
    cudaTriggerProgrammaticLaunchCompletion();             // the scaling may come up meanwhile
    double s = 0.0;
    const uint2 share = share_of(c);
    if (share.x < share.y) {
        int t = tensor_of(c, share.x);
        for (uint32_t g = share.x; g < share.y; ++t) {
            const uint32_t end = min(share.y, c.first[t + 1]);
            const int type = c.type[t];
            const int64_t per = granule_elements(type), from = (int64_t)(g - c.first[t]) * per;
            const int64_t n = min((int64_t)(end - c.first[t]) * per, c.count[t]) - from;
            if (end > g) {
                if (type == SWIGLU_FP32) s += squares(static_cast<const float*>(c.in[t]) + from, n);
                else if (type == SWIGLU_FP16) s += squares(static_cast<const __half*>(c.in[t]) + from, n);
                else s += squares(static_cast<const __nv_bfloat16*>(c.in[t]) + from, n);
            }
            g = end;
        }
    }
    s = cta_sum(s);
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

template <class T>
__device__ __forceinline__ void scale(const T* p, T* o, int64_t n, float f) {
    constexpr int V = 16 / sizeof(T);
    if ((reinterpret_cast<uintptr_t>(p) & 15) != (reinterpret_cast<uintptr_t>(o) & 15)) {
        for (int64_t i = threadIdx.x; i < n; i += kThreads) o[i] = from_f32<T>(to_f32(p[i]) * f);
        return;
    }
    const int64_t head = head_of(p, n);
    const int packs = (int)((n - head) / V);
    const int64_t tail = head + (int64_t)packs * V;
    if (threadIdx.x < head) o[threadIdx.x] = from_f32<T>(to_f32(p[threadIdx.x]) * f);
    if (tail + threadIdx.x < n) o[tail + threadIdx.x] = from_f32<T>(to_f32(p[tail + threadIdx.x]) * f);
    const T* q = p + head;
    uint4* to = reinterpret_cast<uint4*>(o + head);
    constexpr int step = kBlock * kThreads;
    const F2 f2x = f2(f);
    for (int i = (packs + step - 1) / step * step - step; i >= 0; i -= step) {         // the last block first
        uint4 b[kBlock];
        load_block(b, q, i + threadIdx.x, packs);
#pragma unroll
        for (int j = 0; j < kBlock; ++j) {
            const int k = i + threadIdx.x + j * kThreads;
            F2 v[V / 2];
            unpack16<T>(b[j], v);
#pragma unroll
            for (int x = 0; x < V / 2; ++x) v[x] = v[x] * f2x;
            if (k < packs) __stcs(to + k, pack16<T>(v));
        }
    }
}

// The norm from all launches' sums (every CTA, in the same order), then this launch's tensors:
// out = g * min(1, max_norm / (norm + eps)).  Bound by HBM (1.23 GB of bf16 read and written in 381
// us, 6.5 TB/s); from the end of the share, it finds up to an L2's worth of what the norm read last.
template <int N>
__global__ void __launch_bounds__(kThreads, kCtas / kPlanSms) grad_scale_kernel(const __grid_constant__ ClipTable<N> c, const double* sums,
                                                              int num_sums, float max_norm, float eps, float* norm) {
    __shared__ float factor;
    cudaGridDependencySynchronize();         // the sums
    double s = 0.0;
    for (int i = threadIdx.x; i < num_sums; i += kThreads) s += sums[i];
    s = cta_sum(s);
    if (threadIdx.x == 0) {
        const double total = sqrt(s);
        const float f = (float)((double)max_norm / (total + (double)eps));
        factor = f >= 1.f ? 1.f : f;         // a NaN norm gives a NaN factor
        if (norm != nullptr && blockIdx.x == 0) *norm = (float)total;
    }
    __syncthreads();
    const float f = factor;
    const uint2 share = share_of(c);
    if (share.x >= share.y) return;
    int t = tensor_of(c, share.y - 1);
    for (uint32_t end = share.y; end > share.x; --t) {
        const uint32_t g = max(share.x, c.first[t]);
        const int type = c.type[t];
        const int64_t per = granule_elements(type), from = (int64_t)(g - c.first[t]) * per;
        const int64_t n = min((int64_t)(end - c.first[t]) * per, c.count[t]) - from;
        if (end > g && (f != 1.f || c.in[t] != c.out[t])) {        // times 1 in place changes nothing
            if (type == SWIGLU_FP32) scale(static_cast<const float*>(c.in[t]) + from, static_cast<float*>(c.out[t]) + from, n, f);
            else if (type == SWIGLU_FP16) scale(static_cast<const __half*>(c.in[t]) + from, static_cast<__half*>(c.out[t]) + from, n, f);
            else scale(static_cast<const __nv_bfloat16*>(c.in[t]) + from, static_cast<__nv_bfloat16*>(c.out[t]) + from, n, f);
        }
        end = g;
    }
}

int64_t launches_of(int64_t n) { return n <= kMaxTensors ? 1 : (n + kMaxTensors - 1) / kMaxTensors; }

struct ClipCall {
    const void* const* in;
    void* const* out;
    const int64_t* counts;
    const int* types;
    int64_t n;
    float max_norm, eps;
    float* norm;
    double* sums;
    cudaStream_t stream;
};

// Whether an output shares memory with another one, or with an input that is not its own: the scaling's
// CTAs would race on it.  `outs`: room for the n outputs' ranges.
struct Range {
    uintptr_t begin, end;
};
bool outputs_overlap(const ClipCall& a, Range* outs) {
    auto range = [&](const void* p, int64_t i) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        return Range{at, at + (uintptr_t)a.counts[i] * (a.types[i] == SWIGLU_FP32 ? 4 : 2)};
    };
    Range* last = outs;
    for (int64_t i = 0; i < a.n; ++i)
        if (a.counts[i] > 0) *last++ = range(a.out[i], i);
    std::sort(outs, last, [](const Range& p, const Range& q) { return p.begin < q.begin; });
    for (Range* r = outs; r + 1 < last; ++r)
        if (r->end > r[1].begin) return true;
    for (int64_t i = 0; i < a.n; ++i) {
        if (a.counts[i] == 0 || a.in[i] == a.out[i]) continue;
        const Range in = range(a.in[i], i);  // the first output that ends past its begin
        const Range* r = std::partition_point(outs, last, [&](const Range& p) { return p.end <= in.begin; });
        if (r != last && r->begin < in.end) return true;
    }
    return false;
}

// Table of tensors base .. base + N - 1; returns its number of granules.
template <int N>
uint64_t fill_table(ClipTable<N>& c, const ClipCall& a, int64_t base) {
    c.n = (int)(a.n - base < N ? a.n - base : N);
    uint64_t granules = 0;
    for (int i = 0; i < c.n; ++i) {
        c.in[i] = a.in[base + i];
        c.out[i] = a.out ? a.out[base + i] : nullptr;
        c.count[i] = a.counts[base + i];
        c.type[i] = (uint8_t)a.types[base + i];
        c.first[i] = (uint32_t)granules;
        const int64_t per = granule_elements(c.type[i]);
        granules += (uint64_t)((c.count[i] + per - 1) / per);
    }
    c.first[c.n] = (uint32_t)granules;
    return granules;
}

int grid_of(uint64_t granules) { return (int)(granules < (uint64_t)kCtas ? (granules ? granules : 1) : kCtas); }

template <int N>
swiglu_status run_clip(const ClipCall& a) {
    static thread_local ClipTable<N> c;
    const int64_t launches = a.n <= N ? 1 : (a.n + N - 1) / N;
    uint64_t granules = 0;
    int num_sums = 0;
    for (int64_t l = 0; l < launches; ++l) {
        granules = fill_table(c, a, l * N);
        if (granules > 0xffffffffull) return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "clip_grads: the tensors are too large");
        const int grid = grid_of(granules);
        const swiglu_status rc = launch_traced(SWIGLU_KERNEL_GRAD_NORM, a.stream, [&] {
            grad_squares_kernel<N><<<grid, kThreads, 0, a.stream>>>(c, a.sums + num_sums);
            return cudaGetLastError();
        });
        if (rc != SWIGLU_OK) return rc;
        num_sums += grid;
    }
    for (int64_t l = 0; l < (a.out ? launches : 1); ++l) {
        if (!a.out) {                        // only the norm: one CTA, no tensors
            c.n = 0;
            c.first[0] = 0;
            granules = 0;
        } else if (launches > 1) {
            granules = fill_table(c, a, l * N);
        }
        const swiglu_status rc = launch_traced(SWIGLU_KERNEL_GRAD_SCALE, a.stream, [&] {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(grid_of(granules));
            cfg.blockDim = dim3(kThreads);
            cfg.stream = a.stream;
            const double* sums = a.sums;
            float* norm = l == 0 ? a.norm : nullptr;
            return cudaLaunchKernelEx(&cfg, grad_scale_kernel<N>, c, sums, num_sums, a.max_norm, a.eps, norm);
        });
        if (rc != SWIGLU_OK) return rc;
    }
    return SWIGLU_OK;
}

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

size_t swiglu_mlp_clip_grads_workspace_size(int64_t n) {
    return n < 0 ? 0 : (size_t)launches_of(n) * kCtas * sizeof(double);
}

swiglu_status swiglu_mlp_clip_grads(const void* const* in, void* const* out, const int64_t* counts, const int* types,
                                    int64_t n, float max_norm, float eps, float* norm, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    if (n < 0 || (n > 0 && (!in || !counts || !types)) || (!out && !norm) || !workspace)
        return fail(SWIGLU_ERR_INVALID_ARG, "clip_grads: a size is negative or a required pointer is null");
    if (out && (!(max_norm >= 0.f) || !(eps >= 0.f)))
        return fail(SWIGLU_ERR_INVALID_ARG, "clip_grads: max_norm or eps is negative or NaN");
    for (int64_t i = 0; i < n; ++i) {
        const int type = types[i];
        if (type != SWIGLU_BF16 && type != SWIGLU_FP16 && type != SWIGLU_FP32)
            return fail(SWIGLU_ERR_INVALID_ARG, "clip_grads: unknown type");
        if (counts[i] < 0 || (counts[i] > 0 && (!in[i] || (out && !out[i]))))
            return fail(SWIGLU_ERR_INVALID_ARG, "clip_grads: a count is negative or a tensor null");
        if (counts[i] >= (int64_t(1) << 44)) return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "clip_grads: a tensor is too large");
        const uintptr_t bad = (reinterpret_cast<uintptr_t>(in[i]) | (out ? reinterpret_cast<uintptr_t>(out[i]) : 0)) &
                              (type == SWIGLU_FP32 ? 3 : 1);
        if (bad) return fail(SWIGLU_ERR_MISALIGNED, "clip_grads: a tensor is not aligned to its element");
    }
    if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(norm) & 3))
        return fail(SWIGLU_ERR_MISALIGNED, "clip_grads: the workspace is not 16-byte aligned, or norm not 4-byte aligned");
    if (workspace_bytes < swiglu_mlp_clip_grads_workspace_size(n))
        return fail(SWIGLU_ERR_WORKSPACE_TOO_SMALL, "clip_grads: workspace smaller than the size query returns");
    const ClipCall a{in, out, counts, types, n, max_norm, eps, norm, static_cast<double*>(workspace),
                     static_cast<cudaStream_t>(stream)};
    if (out) {
        Range few[kFewTensors];
        const std::unique_ptr<Range[]> many(n > kFewTensors ? new (std::nothrow) Range[n] : nullptr);
        if (n > kFewTensors && !many) return fail(SWIGLU_ERR_CUDA, "clip_grads: no host memory for the tensors' ranges");
        if (outputs_overlap(a, many ? many.get() : few))
            return fail(SWIGLU_ERR_INVALID_ARG, "clip_grads: an output overlaps another one, or an input that is not its own");
    }
    int sms;
    swiglu_status rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    return n <= kFewTensors ? run_clip<kFewTensors>(a) : run_clip<kMaxTensors>(a);
}

}  // extern "C"
