// moe_gate.cu -- the choice of experts from the router's logits and its gradient, and the (token,
// choice) pairs sorted by expert (include/swiglu_tokens.h).
#include <cooperative_groups.h>

#include "rows.cuh"
#include "swiglu_tokens.h"

namespace swiglu {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxExperts = 1024;
constexpr int kGateWarps = 4;

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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A token's logits, lane's own of them in registers (experts lane + 32 i), their largest (0 where none
// is above minus infinity) and the sum of the exponentials.
template <class T, int OWN>
struct Logits {
    float v[OWN], top, sum;
    __device__ __forceinline__ Logits(const Gate& a, int64_t t) {
        const int lane = threadIdx.x & 31;
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            v[i] = lane + 32 * i < a.E ? to_f32(row[lane + 32 * i]) : -INFINITY;
            top = fmaxf(top, v[i]);
        }
        top = warp_max(top);
        if (top == -INFINITY) top = 0.f;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < OWN; ++i) sum += expf(v[i] - top);
        sum = warp_sum(sum);
    }
};

// One warp a token.
template <class T, int OWN>
__global__ void __launch_bounds__(kGateWarps * 32) moe_gate_fwd_kernel(const Gate a) {
    const int64_t t = (int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= a.T) return;
    const Logits<T, OWN> l(a, t);
    uint32_t key[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) key[i] = lane + 32 * i < a.E ? logit_key(l.v[i]) : 0;
    int* ids = a.ids + t * a.k;
    float* gates = a.gates + t * a.k;
    float chosen = 0.f, p;
    int mine;
    for (int j0 = 0; j0 < a.k; j0 += 32) {                 // lane j: choice j0 + j
        const int n = min(32, a.k - j0);
        mine = -1, p = 0.f;
        for (int j = 0; j < n; ++j) {
            uint32_t best = key[0];
            float v = l.v[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < OWN; ++i)
                if (key[i] > best) best = key[i], v = l.v[i], at = i;
            const uint32_t high = __reduce_max_sync(0xffffffffu, best);
            if (high == 0) break;                          // no expert is left
            const int e = __reduce_min_sync(0xffffffffu, best == high ? lane + 32 * at : kMaxExperts);
            v = __shfl_sync(0xffffffffu, v, e & 31);
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                if (e == lane + 32 * i) key[i] = 0;
            if (lane == j) mine = e, p = expf(v - l.top);
        }
        chosen += warp_sum(p);
        if (lane < n) ids[j0 + lane] = mine;
        if (j0 + 32 < a.k) gates[j0 + lane] = mine < 0 ? -1.f : p;      // until all are known
    }
    const float by = a.renorm ? chosen : l.sum;
    auto gate = [&](float e) { return e < 0.f ? 0.f : (isnan(l.sum) ? l.sum : e) / by; };
    const int last = (a.k - 1) / 32 * 32 + lane;
    if (last < a.k) gates[last] = gate(mine < 0 ? -1.f : p);
    for (int j = last - 32; j >= 0; j -= 32) gates[j] = gate(gates[j]);
}

template <class T, int OWN>
__global__ void __launch_bounds__(kGateWarps * 32) moe_gate_bwd_kernel(const Gate a) {
    const int64_t t = (int64_t)blockIdx.x * kGateWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= a.T) return;
    // q and g of choice j0 + lane; its id, -1 where it is no expert
    int id;
    float q, g;
    auto load = [&](int j0) {
        id = j0 + lane < a.k ? a.ids[t * a.k + j0 + lane] : -1, q = g = 0.f;
        if ((unsigned)id < (unsigned)a.E) q = a.gates[t * a.k + j0 + lane], g = a.dgates[t * a.k + j0 + lane];
        else id = -1;
    };
    float s = 0.f;
    for (int j0 = (a.k - 1) / 32 * 32; j0 >= 0; j0 -= 32) {
        load(j0);
        s += q * g;
    }
    s = warp_sum(s);
    T* out = static_cast<T*>(a.dlogits) + t * a.lddl;
    float d[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) d[i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += 32) {
        if (j0 > 0) load(j0);
        const float up = a.renorm ? q * (g - s) : g;
        for (int j = 0; j < min(32, a.k - j0); ++j) {
            const int e = __shfl_sync(0xffffffffu, id, j);
            const float u = __shfl_sync(0xffffffffu, up, j);
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                if (e == lane + 32 * i) d[i] += u;
        }
    }
    if (!a.renorm) {
        const Logits<T, OWN> l(a, t);
#pragma unroll
        for (int i = 0; i < OWN; ++i) d[i] = l.sum == 0.f ? 0.f : expf(l.v[i] - l.top) / l.sum * (d[i] - s);
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i)
        if (lane + 32 * i < a.E) out[lane + 32 * i] = from_f32<T>(d[i]);
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

// Counting sort of the pairs by one cluster.  Each warp has a run of consecutive pairs, 32 at a time,
// and a count for each expert; the counts of all warps, added up over the warps before it and over the
// experts before, are where its first pair of each expert goes.
__global__ void __launch_bounds__(kSortWarps * 32) moe_sort_kernel(const Sort a) {
    extern __shared__ int smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* mine = smem;                      // [E] this CTA's pairs of each expert
    int* base = mine + a.E;                // [E] first row of this CTA's pairs
    int* chunk = base + a.E;               // [32] pairs of 32 experts
    int* hist = chunk + 32;                // [warps][E]
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    int* own = hist + warp * a.E;
    for (int e = lane; e < a.E; e += 32) own[e] = 0;
    __syncwarp();
    const int64_t begin = ((int64_t)rank * warps + warp) * a.per_warp;
    const int64_t end = min(begin + a.per_warp, a.n);
    for (int64_t p0 = begin; p0 < end; p0 += 32) {
        const int e = p0 + lane < end ? a.ids[p0 + lane] : -1;
        const bool in = (unsigned)e < (unsigned)a.E;
        const unsigned same = __match_any_sync(0xffffffffu, in ? e : -1);
        if (in && lane == __ffs(same) - 1) own[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < warps; ++w) {
            const int v = hist[w * a.E + e];
            hist[w * a.E + e] = sum;
            sum += v;
        }
        mine[e] = sum;
    }
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
        for (int w = 0; w < warps; ++w) hist[w * a.E + e] += sum;
    }
    __syncthreads();
    for (int64_t p0 = begin; p0 < end; p0 += 32) {
        const int e = p0 + lane < end ? a.ids[p0 + lane] : -1;
        const bool in = (unsigned)e < (unsigned)a.E;
        const unsigned same = __match_any_sync(0xffffffffu, in ? e : -1);
        const int first = in ? own[e] : -1;
        __syncwarp();
        if (in && lane == __ffs(same) - 1) own[e] = first + __popc(same);
        if (p0 + lane < end) a.pos[p0 + lane] = in ? first + __popc(same & ((1u << lane) - 1)) : -1;
        __syncwarp();
    }
}

// ---------------------------------------------------------------- host side

struct LaunchGate {
    const Gate& a;
    bool bwd;
    cudaStream_t s;
    template <class T, int OWN>
    cudaError_t go() const {
        const unsigned grid = (unsigned)((a.T + kGateWarps - 1) / kGateWarps);
        if (bwd) moe_gate_bwd_kernel<T, OWN><<<grid, kGateWarps * 32, 0, s>>>(a);
        else moe_gate_fwd_kernel<T, OWN><<<grid, kGateWarps * 32, 0, s>>>(a);
        return cudaGetLastError();
    }
    template <class T>
    cudaError_t run() const {
        return a.E <= 32 ? go<T, 1>() : a.E <= 64 ? go<T, 2>() : a.E <= 128 ? go<T, 4>() : a.E <= 256 ? go<T, 8>()
             : a.E <= 512 ? go<T, 16>() : go<T, 32>();
    }
};

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
    const Gate a{logits, nullptr, ids, gates, nullptr, ld, 0, T, (int)E, (int)top_k, renormalize != 0};
    swiglu_status rc = gate_check(a, E, top_k, type);
    if (rc != SWIGLU_OK || T == 0) return rc;
    if (!logits || !ids || !gates) return fail(SWIGLU_ERR_INVALID_ARG, "gate: a required pointer is null");
    if (ld < E) return fail(SWIGLU_ERR_INVALID_ARG, "gate: a row stride is smaller than E");
    if (misaligned(logits, type_bytes(type)) || misaligned(ids, 4) || misaligned(gates, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "gate: a pointer is not aligned to its element");
    int sms;
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_MOE_GATE, s, [&] { return with_type(type, LaunchGate{a, false, s}); });
}

swiglu_status swiglu_moe_gate_bwd(const void* logits, int64_t ld, const int32_t* ids, const float* gates,
                                  const float* dgates, void* dlogits, int64_t lddl, int64_t T, int64_t E,
                                  int64_t top_k, int renormalize, int type, void* stream) {
    const Gate a{logits, dlogits, const_cast<int32_t*>(ids), const_cast<float*>(gates), dgates, ld, lddl, T, (int)E,
                 (int)top_k, renormalize != 0};
    swiglu_status rc = gate_check(a, E, top_k, type);
    if (rc != SWIGLU_OK || T == 0) return rc;
    if ((!logits && !renormalize) || !ids || !gates || !dgates || !dlogits)
        return fail(SWIGLU_ERR_INVALID_ARG, "gate: a required pointer is null");
    if ((!renormalize && ld < E) || lddl < E) return fail(SWIGLU_ERR_INVALID_ARG, "gate: a row stride is smaller than E");
    const size_t n = type_bytes(type);
    if (misaligned(logits, n) || misaligned(dlogits, n) || misaligned(ids, 4) || misaligned(gates, 4) || misaligned(dgates, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "gate: a pointer is not aligned to its element");
    int sms;
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_MOE_GATE, s, [&] { return with_type(type, LaunchGate{a, true, s}); });
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
    const int64_t runs = (pairs + 31) / 32, per_cta = (runs + ctas - 1) / ctas;
    const int warps = (int)(per_cta < 4 ? 4 : per_cta < kSortWarps ? per_cta : kSortWarps);
    const int64_t per_warp = (per_cta + warps - 1) / warps * 32;
    const Sort a{ids, counts, pos, pairs, per_warp, (int)E};
    const size_t smem = ((size_t)(warps + 2) * E + 32) * sizeof(int);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_MOE_SORT, s, [&] {
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(warps * 32);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        return cudaLaunchKernelEx(&cfg, moe_sort_kernel, a);
    });
}

}  // extern "C"
