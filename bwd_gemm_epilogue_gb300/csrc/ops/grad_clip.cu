// grad_clip.cu -- global norm of many gradients and their clipping (include/swiglu_ops.h).
//
// Two launches: sums of squares (one fp64 sum per CTA), then the scaling, whose CTAs each
// add those sums in the same order, so every one of them holds the same norm and no CTA
// waits for another.  The tensors' table travels in the kernels' parameters (no copy, no
// allocation, fit for stream capture); every tensor is cut into chunks of kChunkBytes and
// CTA b takes chunks b, b + gridDim, ...
#include "../host.h"
#include "convert.cuh"
#include "swiglu_ops.h"

namespace swiglu {
namespace {

constexpr int kPlanSms = 152;
constexpr int kThreads = 512;
constexpr int kCtas = kPlanSms * 4;          // persistent CTAs = fp64 sums of one launch
constexpr int kMaxTensors = 768;             // per launch: 22 KB of parameters
constexpr int kFewTensors = 64;              // a second, 2 KB table for the usual few (shorter launches)
constexpr int64_t kChunkBytes = 32768;

template <int N>
struct ClipTable {
    const void* in[N];
    void* out[N];
    int64_t count[N];
    uint32_t first[N + 1];                   // first chunk of each tensor; entry n: the number of chunks
    uint8_t type[N];
    int n;
};

struct Chunk {
    int t;
    int64_t begin, end;                      // elements
};

template <int N>
__device__ __forceinline__ Chunk find_chunk(const ClipTable<N>& c, uint32_t chunk) {
    int lo = 0, hi = c.n;                    // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (c.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    const int64_t per = kChunkBytes / (c.type[lo] == SWIGLU_FP32 ? 4 : 2);
    Chunk k;
    k.t = lo;
    k.begin = (int64_t)(chunk - c.first[lo]) * per;
    k.end = k.begin + per < c.count[lo] ? k.begin + per : c.count[lo];
    return k;
}

// Elements of [begin, end) before the first 16-byte boundary of p.
template <class T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
    const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int64_t)sizeof(T);
    return h < n ? h : n;
}

// This thread's share of the sum of squares of n elements at p.
template <class T, class Acc>
__device__ __forceinline__ Acc squares(const T* p, int64_t n) {
    constexpr int V = 16 / sizeof(T);
    const int64_t head = head_of(p, n);
    Acc s0 = 0, s1 = 0;
    if (threadIdx.x < head) {
        const Acc v = to_f32(p[threadIdx.x]);
        s0 = v * v;
    }
    const T* q = p + head;
    const int packs = (int)((n - head) / V);
#pragma unroll 4
    for (int i = threadIdx.x; i < packs; i += kThreads) {
        float v[V];
        load_pack<T, V>(q + (int64_t)i * V).unpack(v);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const Acc a = v[j], b = v[j + 1];
            s0 += a * a;
            s1 += b * b;
        }
    }
    const int64_t tail = head + (int64_t)packs * V;
    if (tail + threadIdx.x < n) {
        const Acc v = to_f32(p[tail + threadIdx.x]);
        s1 += v * v;
    }
    return s0 + s1;
}

template <class T>
__device__ __noinline__ double squares_again(const T* p, int64_t n) {
    return squares<T, double>(p, n);
}

// In fp32, and once more in fp64 where that overflowed (finite elements above 1.8e19 do).
template <class T>
__device__ __forceinline__ double chunk_squares(const T* p, int64_t n) {
    const float s = squares<T, float>(p, n);
    return isinf(s) ? squares_again(p, n) : (double)s;
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

template <int N>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ ClipTable<N> c, double* sums) {
    double s = 0.0;
    for (uint32_t k = blockIdx.x; k < c.first[c.n]; k += gridDim.x) {
        const Chunk u = find_chunk(c, k);
        const int type = c.type[u.t];
        const int64_t n = u.end - u.begin;
        if (type == SWIGLU_FP32) s += chunk_squares(static_cast<const float*>(c.in[u.t]) + u.begin, n);
        else if (type == SWIGLU_FP16) s += chunk_squares(static_cast<const __half*>(c.in[u.t]) + u.begin, n);
        else s += chunk_squares(static_cast<const __nv_bfloat16*>(c.in[u.t]) + u.begin, n);
    }
    s = cta_sum(s);
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

template <class T>
__device__ __forceinline__ void scale_chunk(const T* p, T* o, int64_t n, float f) {
    constexpr int V = 16 / sizeof(T);
    if ((reinterpret_cast<uintptr_t>(p) & 15) != (reinterpret_cast<uintptr_t>(o) & 15)) {
        for (int64_t i = threadIdx.x; i < n; i += kThreads) o[i] = from_f32<T>(to_f32(p[i]) * f);
        return;
    }
    const int64_t head = head_of(p, n);
    if (threadIdx.x < head) o[threadIdx.x] = from_f32<T>(to_f32(p[threadIdx.x]) * f);
    const int packs = (int)((n - head) / V);
#pragma unroll 4
    for (int i = threadIdx.x; i < packs; i += kThreads) {
        float v[V];
        load_pack<T, V>(p + head + (int64_t)i * V).unpack(v);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= f;
        store_pack<T, V>(o + head + (int64_t)i * V, v);
    }
    const int64_t tail = head + (int64_t)packs * V;
    if (tail + threadIdx.x < n) o[tail + threadIdx.x] = from_f32<T>(to_f32(p[tail + threadIdx.x]) * f);
}

// The norm from all launches' sums (every CTA, in the same order), then this launch's tensors.
template <int N>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ ClipTable<N> c, const double* sums,
                                                              int num_sums, float max_norm, float eps, float* norm) {
    __shared__ float factor;
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
    const uint32_t chunks = c.first[c.n];
    for (uint32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
        const Chunk u = find_chunk(c, k);
        const int type = c.type[u.t];
        const int64_t n = u.end - u.begin;
        if (type == SWIGLU_FP32)
            scale_chunk(static_cast<const float*>(c.in[u.t]) + u.begin, static_cast<float*>(c.out[u.t]) + u.begin, n, f);
        else if (type == SWIGLU_FP16)
            scale_chunk(static_cast<const __half*>(c.in[u.t]) + u.begin, static_cast<__half*>(c.out[u.t]) + u.begin, n, f);
        else
            scale_chunk(static_cast<const __nv_bfloat16*>(c.in[u.t]) + u.begin,
                        static_cast<__nv_bfloat16*>(c.out[u.t]) + u.begin, n, f);
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

// Table of tensors base .. base + N - 1; returns its number of chunks.
template <int N>
uint64_t fill_table(ClipTable<N>& c, const ClipCall& a, int64_t base) {
    c.n = (int)(a.n - base < N ? a.n - base : N);
    uint64_t chunks = 0;
    for (int i = 0; i < c.n; ++i) {
        c.in[i] = a.in[base + i];
        c.out[i] = a.out ? a.out[base + i] : nullptr;
        c.count[i] = a.counts[base + i];
        c.type[i] = (uint8_t)a.types[base + i];
        c.first[i] = (uint32_t)chunks;
        const int64_t per = kChunkBytes / (c.type[i] == SWIGLU_FP32 ? 4 : 2);
        chunks += (uint64_t)((c.count[i] + per - 1) / per);
    }
    c.first[c.n] = (uint32_t)chunks;
    return chunks;
}

int grid_of(uint64_t chunks) { return (int)(chunks < (uint64_t)kCtas ? (chunks ? chunks : 1) : kCtas); }

template <int N>
swiglu_status run_clip(const ClipCall& a) {
    static thread_local ClipTable<N> c;
    const int64_t launches = a.n <= N ? 1 : (a.n + N - 1) / N;
    uint64_t chunks = 0;
    int num_sums = 0;
    for (int64_t l = 0; l < launches; ++l) {
        chunks = fill_table(c, a, l * N);
        if (chunks > 0xffffffffull - kCtas) return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "clip_grads: the tensors are too large");
        const int grid = grid_of(chunks);
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
            chunks = 0;
        } else if (launches > 1) {
            chunks = fill_table(c, a, l * N);
        }
        const swiglu_status rc = launch_traced(SWIGLU_KERNEL_GRAD_SCALE, a.stream, [&] {
            grad_scale_kernel<N><<<grid_of(chunks), kThreads, 0, a.stream>>>(c, a.sums, num_sums, a.max_norm, a.eps,
                                                                            l == 0 ? a.norm : nullptr);
            return cudaGetLastError();
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
    int sms;
    swiglu_status rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    const ClipCall a{in, out, counts, types, n, max_norm, eps, norm, static_cast<double*>(workspace),
                     static_cast<cudaStream_t>(stream)};
    return n <= kFewTensors ? run_clip<kFewTensors>(a) : run_clip<kMaxTensors>(a);
}

}  // extern "C"
