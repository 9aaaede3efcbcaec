// moe_routed.cu -- a whole mixture-of-experts layer for a few tokens (include/swiglu_moe.h,
// swiglu_moe_routed_fwd): router, choice of experts, the chosen experts' SwiGLU blocks and
// the weighted sum per token.
//
// With at most 64 tokens the work is to read the chosen experts' weights once; the tokens
// that share an expert share that read.  Three launches, and nothing on the host depends
// on the routing: the kernels read the chosen ids and divide what was chosen among
// themselves.
//
//   route  one thread-block cluster per token: logits, softmax, top-k
//   up     per chosen expert, 8 hidden units: left and gate rows of W1 against the
//          expert's tokens, h = left * silu(gate) -> h [T * k, H] bf16 in the workspace
//   down   16 output columns of every token: W2 rows of all chosen experts against h,
//          weighted by the gates and added in registers and shared memory
//
// Weights go from global memory straight into the registers of mma.m16n8k16 (A, 16 weight
// rows) and are never staged: a lane's 16-byte load holds 8 consecutive k of one row, and
// since a dot product does not care for the order of k, those 8 feed two MMAs (4 k each)
// as long as the tokens' operand B is loaded with the same assignment.  A warp keeps
// kDepth steps of 64 k (2 KB of weights each) in flight.
#include <cooperative_groups.h>

#include "../host.h"
#include "convert.cuh"
#include "swiglu_moe.h"

namespace swiglu {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanSms = 152;
constexpr int kMaxTokens = 64;
constexpr int kMaxTop = 16;
constexpr int kMaxExperts = 682;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kCtas = kPlanSms * 2;          // two CTAs an SM: 16 warps x kDepth x 2 KB in flight
constexpr int kDepth = 4;

struct Routed {
    const __nv_bfloat16 *x, *W1, *W2, *r;
    const void* Wr;
    __nv_bfloat16 *y, *h;
    int* ids;
    float* gates;
    int T, E, D, H, Dout, k, renorm, wr32;
};

// ---------------------------------------------------------------- route

// 8 values of a row at p as fp32.
__device__ __forceinline__ void load8(float* o, const __nv_bfloat16* p) {
    load_pack<__nv_bfloat16, 8>(p).unpack(o);
}
__device__ __forceinline__ void load8(float* o, const float* p) {
    load_pack<float, 4>(p).unpack(o);
    load_pack<float, 4>(p + 4).unpack(o + 4);
}

// Order-preserving key of a logit: larger logit, larger key; NaN lowest.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (isnan(v)) return 0;
    const uint32_t u = __float_as_uint(v + 0.f);           // -0 counts as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One cluster per token; CTA rank c computes the logits of experts c * kWarps + warp,
// + cluster size * kWarps, ...; the first CTA's first warp chooses.
template <class W>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(const Routed a) {
    __shared__ float logits[kMaxExperts];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int t = blockIdx.x / ctas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* all = cluster.map_shared_rank(logits, 0);
    const __nv_bfloat16* x = a.x + (int64_t)t * a.D;
    for (int e = rank * kWarps + warp; e < a.E; e += ctas * kWarps) {
        const W* w = static_cast<const W*>(a.Wr) + (int64_t)e * a.D;
        float s = 0.f;
#pragma unroll 4
        for (int c = lane * 8; c < a.D; c += 256) {
            float xv[8], wv[8];
            load8(xv, x + c);
            load8(wv, w + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += xv[j] * wv[j];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) all[e] = s;
    }
    cluster.sync();
    if (rank != 0 || warp != 0) return;

    float top = -INFINITY, sum = 0.f;
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, logits[e]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int e = lane; e < a.E; e += 32) sum += expf(logits[e] - top);      // a NaN logit makes every gate NaN
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    uint32_t taken = 0;                                    // bit i: expert lane + 32 i
    int mine = 0;
    float weight = 0.f, chosen = 0.f;
    for (int j = 0; j < a.k; ++j) {
        uint32_t key = 0;
        int best = kMaxExperts;
        for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
            if (taken >> i & 1) continue;
            const uint32_t q = logit_key(logits[e]);
            if (best == kMaxExperts || q > key) key = q, best = e;
        }
        const uint32_t high = __reduce_max_sync(0xffffffffu, best < kMaxExperts ? key : 0);
        const int e = __reduce_min_sync(0xffffffffu, best < kMaxExperts && key == high ? best : kMaxExperts);
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        const float p = expf(logits[e] - top);
        chosen += p;
        if (lane == j) mine = e, weight = p;
    }
    if (isnan(sum)) weight = sum;
    if (lane < a.k) {
        a.ids[t * a.k + lane] = mine;
        a.gates[t * a.k + lane] = weight / (a.renorm ? chosen : sum);
    }
}

// ---------------------------------------------------------------- what was chosen

// Shared by the up and the down kernel: for every expert the tokens that chose it (a bit
// each), and the experts chosen at all, in ascending order.
struct Chosen {
    unsigned long long tokens[kMaxExperts];
    short expert[kMaxExperts + 2];
    short ids[kMaxTokens * kMaxTop];
    int count;
};

__device__ __forceinline__ void read_choice(Chosen& c, const Routed& a) {
    for (int e = threadIdx.x; e < a.E; e += kThreads) c.tokens[e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < a.T * a.k; p += kThreads) {
        const int e = a.ids[p];
        c.ids[p] = (short)e;
        atomicOr(&c.tokens[e], 1ull << (p / a.k));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + threadIdx.x;
            const bool in = e < a.E && c.tokens[e] != 0;
            const unsigned m = __ballot_sync(0xffffffffu, in);
            if (in) c.expert[n + __popc(m & ((1u << threadIdx.x) - 1))] = (short)e;
            n += __popc(m);
        }
        if (threadIdx.x == 0) c.count = n;
    }
    __syncthreads();
}

// This warp's list of expert e's (token, choice) pairs, in token order: pair = token * k + j.
// Entries past the count repeat the last pair (their columns are computed and dropped).
__device__ __forceinline__ int list_pairs(short* list, const Chosen& c, const Routed& a, int e) {
    const int lane = threadIdx.x & 31;
    const unsigned long long m = c.tokens[e];
    const int n = __popcll(m);
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int t = lane + 32 * half;
        if (m >> t & 1) {
            int j = 0;
            while (c.ids[t * a.k + j] != e) ++j;
            const int at = __popcll(m & ((1ull << t) - 1));
            list[at] = (short)(t * a.k + j);
            if (at == n - 1)
                for (int q = n; q < kMaxTokens; ++q) list[q] = (short)(t * a.k + j);
        }
    }
    __syncwarp();
    return n;
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ uint4 load_weights(const __nv_bfloat16* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc += the products of 16 weight rows with NT * 8 token rows over k steps [s0, s1) of 64.
// Lane (g, q) = (lane / 4, lane % 4): w0, w1 are its weight rows g and g + 8; token row
// n * 8 + g starts at b + off[n].  acc[n]: rows g and g + 8 x tokens n * 8 + 2 q, + 1.
template <int NT>
__device__ __forceinline__ void products(float (*acc)[4], const __nv_bfloat16* w0, const __nv_bfloat16* w1,
                                         const __nv_bfloat16* b, const int* off, int s0, int s1, int K) {
    const int q = (threadIdx.x & 3) * 8;
    uint4 w[kDepth][4];
    auto load = [&](int d, int s) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const int c = s * 64 + q;
        const bool in0 = s < s1 && c < K, in1 = s < s1 && c + 32 < K;
        w[d][0] = in0 ? load_weights(w0 + c) : zero;
        w[d][1] = in0 ? load_weights(w1 + c) : zero;
        w[d][2] = in1 ? load_weights(w0 + c + 32) : zero;
        w[d][3] = in1 ? load_weights(w1 + c + 32) : zero;
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(d, s0 + d);
    for (int s = s0; s < s1; s += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (s + d < s1) {
                const int c = (s + d) * 64 + q;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    const uint4 u = c < K ? *reinterpret_cast<const uint4*>(b + off[n] + c) : zero;
                    const uint4 v = c + 32 < K ? *reinterpret_cast<const uint4*>(b + off[n] + c + 32) : zero;
                    mma(acc[n], w[d][0].x, w[d][1].x, w[d][0].y, w[d][1].y, u.x, u.y);
                    mma(acc[n], w[d][0].z, w[d][1].z, w[d][0].w, w[d][1].w, u.z, u.w);
                    mma(acc[n], w[d][2].x, w[d][3].x, w[d][2].y, w[d][3].y, v.x, v.y);
                    mma(acc[n], w[d][2].z, w[d][3].z, w[d][2].w, w[d][3].w, v.z, v.w);
                }
                load(d, s + d + kDepth);
            }
        }
    }
}

// products() over the number of 8-token tiles that n tokens take.
__device__ __forceinline__ void products_of(int n, float (*acc)[4], const __nv_bfloat16* w0, const __nv_bfloat16* w1,
                                            const __nv_bfloat16* b, const int* off, int s0, int s1, int K) {
    if (n <= 8) products<1>(acc, w0, w1, b, off, s0, s1, K);
    else if (n <= 16) products<2>(acc, w0, w1, b, off, s0, s1, K);
    else if (n <= 32) products<4>(acc, w0, w1, b, off, s0, s1, K);
    else products<8>(acc, w0, w1, b, off, s0, s1, K);
}

// Unit = 8 hidden units of a chosen expert: MMA rows 0..7 are their left rows of W1, rows
// 8..15 the gate rows of the same units, so a lane ends with left and gate of its unit.
// A unit's k range is split over `split` warps of the CTA, whose sums meet in shared memory.
__global__ void __launch_bounds__(kThreads, 2) moe_up_kernel(const Routed a) {
    __shared__ Chosen chosen;
    __shared__ short lists[kWarps][kMaxTokens];
    __shared__ float part[kWarps][32][33];
    read_choice(chosen, a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int groups = a.H / 8, units = chosen.count * groups, steps = (a.D + 63) / 64;
    // the split whose last round wastes least: time of a launch in whole units
    int split = 1;
    float best = INFINITY;
    for (int s = 1; s <= kWarps; s *= 2) {
        const int per = gridDim.x * (kWarps / s);
        const float cost = (float)((units + per - 1) / per) / (float)s * (1.f + 0.01f * s);
        if (cost < best) best = cost, split = s;
    }
    const int sub = warp / split, piece = warp % split, subs = kWarps / split;
    const int s0 = steps * piece / split, s1 = steps * (piece + 1) / split;
    const int rounds = (units + gridDim.x * subs - 1) / (gridDim.x * subs);
    int last = -1, n = 0;
    int off[8];
    for (int r = 0; r < rounds; ++r) {
        const int u = (r * subs + sub) * gridDim.x + blockIdx.x;
        const bool on = u < units;
        float acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
        const int unit = on ? u % groups * 8 + g : 0;
        if (on) {
            const int e = chosen.expert[u / groups];
            if (e != last) {
                last = e;
                n = list_pairs(lists[warp], chosen, a, e);
#pragma unroll
                for (int i = 0; i < 8; ++i) off[i] = lists[warp][i * 8 + g] / a.k * a.D;
            }
            const __nv_bfloat16* w0 = a.W1 + ((int64_t)e * 2 * a.H + unit) * a.D;
            products_of(n, acc, w0, w0 + (int64_t)a.H * a.D, a.x, off, s0, s1, a.D);
        }
        if (split > 1) {
            if (piece > 0 && on) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i * 8 < n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[warp][i * 4 + j][lane] = acc[i][j];
            }
            __syncthreads();
            if (piece == 0 && on) {
                for (int p = 1; p < split; ++p)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i * 8 < n)
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[i][j] += part[warp + p][i * 4 + j][lane];
            }
            __syncthreads();
        }
        if (on && piece == 0) {
            // h is rounded to bf16 once, for the down product's MMA; left and gate stay fp32
#pragma unroll
            for (int i = 0; i < 8; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = i * 8 + 2 * q + j;
                    if (col < n) {
                        const float left = acc[i][j], gate = acc[i][2 + j];
                        a.h[(int64_t)lists[warp][col] * a.H + unit] =
                            __float2bfloat16_rn(left * (gate / (1.f + __expf(-gate))));
                    }
                }
            }
        }
    }
}

// Cluster of CTAs = 16 output columns.  The steps of all chosen experts, one after the
// other, are divided evenly over the cluster's warps; a warp adds each expert's sums,
// times the gates, into its own fp32 tile [T][16], and the tiles are added in warp order.
__global__ void __launch_bounds__(kThreads, 2) moe_down_kernel(const Routed a) {
    __shared__ Chosen chosen;
    __shared__ short lists[kWarps][kMaxTokens];
    extern __shared__ float sums[];                        // [kWarps][T][16]
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    read_choice(chosen, a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int row0 = blockIdx.x / ctas * 16, steps = (a.H + 63) / 64;
    float* mine = sums + warp * a.T * 16;
    for (int i = lane; i < a.T * 16; i += 32) mine[i] = 0.f;
    const int64_t total = (int64_t)chosen.count * steps;
    const int workers = ctas * kWarps, me = rank * kWarps + warp;
    int64_t at = total * me / workers;
    const int64_t end = total * (me + 1) / workers;
    const int r1 = row0 + g + 8 < a.Dout ? row0 + g + 8 : row0 + g;     // Dout is a multiple of 8
    while (at < end) {
        const int e = chosen.expert[at / steps];
        const int s0 = (int)(at % steps);
        const int s1 = (int)(end - at < steps - s0 ? s0 + (end - at) : steps);
        const int n = list_pairs(lists[warp], chosen, a, e);
        int off[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) off[i] = lists[warp][i * 8 + g] * a.H;
        float acc[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
        const __nv_bfloat16* w = a.W2 + (int64_t)e * a.Dout * a.H;
        products_of(n, acc, w + (int64_t)(row0 + g) * a.H, w + (int64_t)r1 * a.H, a.h, off, s0, s1, a.H);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = i * 8 + 2 * q + j;
                if (col < n) {
                    const int p = lists[warp][col];
                    const float gate = a.gates[p];
                    float* o = mine + p / a.k * 16 + g;
                    o[0] += gate * acc[i][j];
                    o[8] += gate * acc[i][2 + j];
                }
            }
        }
        at += s1 - s0;
    }
    cluster.sync();
    if (rank == 0) {
        for (int i = threadIdx.x; i < a.T * 16; i += kThreads) {
            const int t = i / 16, col = row0 + i % 16;
            float v = 0.f;
            for (int c = 0; c < ctas; ++c) {
                const float* s = cluster.map_shared_rank(sums, c);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += s[w * a.T * 16 + i];
            }
            if (col < a.Dout) {
                const int64_t o = (int64_t)t * a.Dout + col;
                if (a.r) v += to_f32(a.r[o]);
                a.y[o] = __float2bfloat16_rn(v);
            }
        }
    }
    cluster.sync();                                        // the sums stay until rank 0 has read them
}

// ---------------------------------------------------------------- host side

bool width_ok(int64_t v) { return v > 0 && v % 8 == 0 && v < (int64_t(1) << 24); }

cudaError_t launch_clusters(void (*kernel)(Routed), const Routed& a, int clusters, int size, size_t smem,
                            cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(clusters * size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

size_t swiglu_moe_routed_fwd_workspace_size(int64_t T, int64_t H, int64_t top_k) {
    if (T <= 0 || H <= 0 || top_k <= 0) return 0;
    return ((size_t)T * (size_t)top_k * (size_t)H * 2 + 255) & ~size_t(255);
}

swiglu_status swiglu_moe_routed_fwd(const void* x, const void* Wr, const void* W1, const void* W2,
                                    const void* residual, void* y, int32_t* ids, float* gates, int64_t T, int64_t E,
                                    int64_t D, int64_t H, int64_t Dout, int64_t top_k, int renormalize,
                                    int router_fp32, void* workspace, size_t workspace_bytes, void* stream) {
    if (T < 0 || E <= 0 || D <= 0 || H <= 0 || Dout <= 0 || top_k <= 0 || top_k > E)
        return fail(SWIGLU_ERR_INVALID_ARG, "routed layer: a size is negative or zero, or top_k above E");
    if (T > kMaxTokens || E > kMaxExperts || top_k > kMaxTop || !width_ok(D) || !width_ok(H) || !width_ok(Dout))
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "routed layer: needs T <= 64, E <= 682, top_k <= 16 and widths that are multiples of 8 below 2^24");
    if (T == 0) return SWIGLU_OK;
    if (T * top_k * H >= (int64_t(1) << 31)) return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "routed layer: T * top_k * H must stay below 2^31");
    if (!x || !Wr || !W1 || !W2 || !y || !ids || !gates || !workspace)
        return fail(SWIGLU_ERR_INVALID_ARG, "routed layer: a required pointer is null");
    if (!aligned16(x) || !aligned16(Wr) || !aligned16(W1) || !aligned16(W2) || !aligned16(residual) || !aligned16(y) ||
        !aligned16(workspace) || (reinterpret_cast<uintptr_t>(ids) & 3) || (reinterpret_cast<uintptr_t>(gates) & 3))
        return fail(SWIGLU_ERR_MISALIGNED, "routed layer: a pointer is not 16-byte aligned (ids, gates: 4)");
    if (workspace_bytes < swiglu_moe_routed_fwd_workspace_size(T, H, top_k))
        return fail(SWIGLU_ERR_WORKSPACE_TOO_SMALL, "routed layer: workspace smaller than the size query returns");
    int sms;
    swiglu_status rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    typedef const __nv_bfloat16* In;
    const Routed a{(In)x, (In)W1, (In)W2, (In)residual, Wr, (__nv_bfloat16*)y, (__nv_bfloat16*)workspace, ids, gates,
                   (int)T, (int)E, (int)D, (int)H, (int)Dout, (int)top_k, renormalize != 0, router_fp32 != 0};
    // route: up to 8 CTAs of 8 warps share a token's experts
    const int route_ctas = E <= 8 ? 1 : E <= 16 ? 2 : E <= 32 ? 4 : 8;
    rc = launch_traced(SWIGLU_KERNEL_MOE_ROUTE, s, [&] {
        return launch_clusters(router_fp32 ? moe_route_kernel<float> : moe_route_kernel<__nv_bfloat16>, a, (int)T,
                               route_ctas, 0, s);
    });
    if (rc != SWIGLU_OK) return rc;
    rc = launch_traced(SWIGLU_KERNEL_MOE_UP, s, [&] {
        moe_up_kernel<<<kCtas, kThreads, 0, s>>>(a);
        return cudaGetLastError();
    });
    if (rc != SWIGLU_OK) return rc;
    // down: the largest cluster that leaves the CTAs resident at once
    const int tiles = (int)((Dout + 15) / 16);
    int size = 1;
    while (size < 8 && tiles * size * 2 <= kCtas) size *= 2;
    return launch_traced(SWIGLU_KERNEL_MOE_DOWN, s, [&] {
        return launch_clusters(moe_down_kernel, a, tiles, size, (size_t)kWarps * T * 16 * sizeof(float), s);
    });
}

}  // extern "C"
