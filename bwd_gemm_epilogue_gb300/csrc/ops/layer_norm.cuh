// layer_norm.cuh -- what the layer norm's two directions share: how rows lie in 16-byte packs,
// gamma and beta in shared memory, sums over a row, and the plan of a launch.
#pragma once

#include "../host.h"
#include "convert.cuh"
#include "swiglu_ops.h"

namespace swiglu {
namespace {

constexpr int kPlanSms = 152;      // grids are planned for the GB300, so that the workspace query sees no device
constexpr int kMaxThreads = 512;   // the forms for rows too wide for registers
constexpr size_t kSmem = 227 * 1024;

// ---------------------------------------------------------------- 16-byte packs of a row

template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// Rows that do not start on 16-byte boundaries, or end off them, but lie alike in every tensor:
// pack k is then the aligned 16 bytes with the columns k * kVec - m ... of the row, where the row
// starts m elements into its first pack.  All that has to be told apart are the first and the
// last pack (their other elements belong to the neighbouring rows), and the parameters, which do
// not start inside a pack, go through shared memory.
template <class T>
__device__ __forceinline__ int into_pack(const void* base, int64_t row, int64_t ld) {
    return (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * ld) & 15) / sizeof(T));
}

// The elements of the pack that starts at column `first` which are the row's, others 0.
template <class T>
__device__ __forceinline__ uint4 row_elements(uint4 v, int first, int D) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) {
        const uint32_t bits = sizeof(T) == 4 ? ~0u : 0xffffu << (j % per * 16);
        if ((unsigned)(first + j) >= (unsigned)D) w[j / per] &= ~bits;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// They alone, loaded and stored one by one; `row`: column 0.
template <class T>
__device__ __forceinline__ uint4 load_edge(const T* row, int first, int D) {
    uint32_t w[4] = {0, 0, 0, 0};
    constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) {
        if ((unsigned)(first + j) < (unsigned)D) {
            if constexpr (sizeof(T) == 4) w[j] = *reinterpret_cast<const uint32_t*>(row + first + j);
            else w[j / per] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + first + j) << (j % per * 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <class T>
__device__ __forceinline__ void store_edge(T* row, int first, int D, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) {
        if ((unsigned)(first + j) < (unsigned)D) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(row + first + j) = w[j];
            else *reinterpret_cast<uint16_t*>(row + first + j) = (uint16_t)(w[j / per] >> (j % per * 16));
        }
    }
}

__device__ __forceinline__ uint4 load_smem(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store_smem(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// gamma or beta as fp32 in shared memory: the first 16 bytes of every pack's values, then
// (16-bit rows) the second 16 bytes of every pack's, so that a warp's 16-byte reads touch
// every bank once.
__host__ __device__ constexpr int padded(int D) { return (D + 7) / 8 * 8; }

template <class T>
__device__ __forceinline__ int staged_at(int c, int width) {
    return sizeof(T) == 4 ? c : (c & 4 ? width / 2 : 0) + (c >> 3) * 4 + (c & 3);
}

// 16 bytes of W at a time, several in flight (one value at a time, 5003 columns of two took 10 us).
template <class T, class W>
__device__ __forceinline__ void stage_values(float* to, const W* p, int D, int m, int width, int t, int threads) {
    constexpr int V = 16 / (int)sizeof(W);
    const int whole = (reinterpret_cast<uintptr_t>(p) & 15) == 0 ? D / V : 0;
#pragma unroll 4
    for (int k = t; k < whole; k += threads) {
        F2 f[V / 2];
        unpack16<W>(reinterpret_cast<const uint4*>(p)[k], f);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const float2 v = split(f[j]);
            to[staged_at<T>(k * V + 2 * j + m, width)] = v.x;
            to[staged_at<T>(k * V + 2 * j + 1 + m, width)] = v.y;
        }
    }
#pragma unroll 8
    for (int c = whole * V + t; c < D; c += threads) to[staged_at<T>(c + m, width)] = to_f32(p[c]);
}

// By `threads` threads of which this is number t.  The packs start m columns before the row;
// `width`: the places of `to`, whole packs; those outside the row are zeros.
template <class T>
__device__ __forceinline__ void stage_param(float* to, const void* p, int gf32, int D, int m, int width, float none, int t,
                                            int threads) {
    if (p == nullptr) {
        for (int c = t; c < D; c += threads) to[staged_at<T>(c + m, width)] = none;
    } else if (gf32) {
        stage_values<T>(to, static_cast<const float*>(p), D, m, width, t, threads);
    } else {
        stage_values<T>(to, static_cast<const T*>(p), D, m, width, t, threads);
    }
    if (t < m) to[staged_at<T>(t, width)] = 0.f;
    for (int c = D + m + t; c < width; c += threads) to[staged_at<T>(c, width)] = 0.f;
}

// Pack k of one, as pairs.
template <class T>
__device__ __forceinline__ void load_staged(F2* o, uint32_t p, int k, int width) {
    unpack16<float>(load_smem(p + k * 16), o);
    if constexpr (sizeof(T) == 2) unpack16<float>(load_smem(p + width * 2 + k * 16), o + 2);
}

// One value of gamma or beta.
template <class T>
__device__ __forceinline__ float param(const void* p, int gf32, int col, float none, T*) {
    return p == nullptr ? none : gf32 && sizeof(T) != 4 ? static_cast<const float*>(p)[col] : to_f32(static_cast<const T*>(p)[col]);
}

// Whether pack k = q * lanes + lane is the row's, which ends at element `end` of its packs: the
// plan gives a row ceil(packs / lanes) packs a thread, so only the last one can be past it.
template <class T, int NV>
__device__ __forceinline__ bool in_row(int q, int k, int end) {
    return q < NV - 1 || k * kVec<T> < end;
}

// EDGE: whether pack k = q * lanes + lane is the first or the last, with elements that are not the
// row's (the last one has q >= NV - 2).
template <class T, int NV>
__device__ __forceinline__ bool on_edge(int q, int k, int m, int end) {
    return (q == 0 && k == 0 && m > 0) || (q >= NV - 2 && k * kVec<T> + kVec<T> > end);
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

// A thread's sum over a row wider than the registers hold, up to half a million elements: runs of a
// pack or of kRun single elements in fp32, whose sums are added with the rounding error of each
// addition kept (Knuth's two-sum), so it is off by one run's roundings however long the row.  (A plain
// running sum of 2^24 columns of 1.1 put the mean off by 1e-4, and with it every difference from it.)
constexpr int kRun = 32;
struct LongSum {
    float sum = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float t = sum + v, z = t - sum;
        lost += (sum - (t - z)) + (v - z);
        sum = t;
    }
    __device__ __forceinline__ float value() const {       // infinite sums have no error to speak of
        const float v = sum + lost;
        return v == v ? v : sum;
    }
};

// Rows off 16-byte boundaries, element by element (those that lie differently in the call's tensors,
// and those that shifted packs do not pay for): thread t of a
// row's THREADS has columns t + i * THREADS, i < kCols, whose offsets are constants; kCols
// loads a thread keep enough bytes in flight, and a warp still reads 64 or 128 bytes in a row.
constexpr int kCols = 16;

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

// ---------------------------------------------------------------- host side

// How a launch covers its rows: `nv` packs a thread, `lanes` threads a row, `groups` rows a
// CTA at a time.
struct NormPlan {
    int nv, lanes, groups;
    int threads() const { return lanes * groups; }
};

// Widest packs of a row: they may start up to a pack less an element before it.
inline int64_t reach(int64_t D, int size, bool edge) { return edge ? D + 16 / size - 1 : D; }

inline NormPlan norm_plan(int64_t width, int size, int packs, int threads) {
    NormPlan p;
    const int64_t all = (width * size + 15) / 16;
    p.lanes = (int)((all + packs * 32 - 1) / (packs * 32) * 32);
    p.nv = (int)((all + p.lanes - 1) / p.lanes);
    p.groups = threads / p.lanes > 1 ? threads / p.lanes : 1;
    return p;
}

// Rows element by element: THREADS of a row, and (backward) workers that share the rows; each
// worker has a partial plane, so the wider the row, the fewer.  Wider than 8192: two passes.
inline int narrow_threads(int64_t D) { return D <= 32 * kCols ? 32 : D <= 128 * kCols ? 128 : 512; }
constexpr int64_t kNarrowWidth = 512 * kCols;
// Bytes an element of `type` takes; 0 for an unknown type.
inline int type_bytes(int type) { return type == SWIGLU_FP32 ? 4 : type == SWIGLU_BF16 || type == SWIGLU_FP16 ? 2 : 0; }

inline bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// How a call's rows lie: every base, row stride and the width on 16-byte boundaries (kWhole), or
// off them but each row alike in all tensors (kEdge), or neither (kApart).  A row of less than
// kLeastEdge bytes counts as kApart: most of its packs would be edges.
enum Lie { kWhole, kEdge, kApart };
constexpr int64_t kLeastEdge = 128;
struct Rows16 {
    int size, bits = 0, base = -1, ld16 = -1;
    bool alike = true;
    void add(const void* p, int64_t ld) {
        if (!p) return;
        const int b = (int)(reinterpret_cast<uintptr_t>(p) & 15), l = (int)((ld * size) & 15);
        bits |= b | l;
        if (base < 0) base = b, ld16 = l;
        alike = alike && b == base && l == ld16;
    }
    Lie lie(int64_t D) const {
        if (bits == 0 && D * size % 16 == 0) return kWhole;
        return alike && D * size >= kLeastEdge ? kEdge : kApart;
    }
};

// f.run<T>() for the run-time type.
template <class F>
cudaError_t with_type(int type, const F& f) {
    if (type == SWIGLU_FP32) return f.template run<float>();
    if (type == SWIGLU_FP16) return f.template run<__half>();
    return f.template run<__nv_bfloat16>();
}

// Past 48 KB, of which the kernels' own arrays take less than 1 KB, a launch has to be allowed.
template <class K>
cudaError_t allow_smem(K kern, size_t bytes) {
    return bytes <= 47 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

inline swiglu_status norm_check(int64_t M, int64_t D, int type, int param_type) {
    if (M < 0 || D <= 0) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a size is negative or zero");
    if (M >= (int64_t(1) << 31) || D >= (int64_t(1) << 28))
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "layer norm: M must stay below 2^31 and D below 2^28");
    if (type_bytes(type) == 0 || (param_type != type && param_type != SWIGLU_FP32))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: unknown type, or parameters of neither the rows' type nor fp32");
    return SWIGLU_OK;
}

}  // namespace
}  // namespace swiglu
