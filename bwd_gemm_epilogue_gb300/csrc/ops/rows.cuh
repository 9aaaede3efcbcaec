// rows.cuh -- rows of a tensor in 16-byte packs, what the operators on rows of bf16, fp16 and fp32
// have in common.
#pragma once

#include "launch.cuh"
#include "convert.cuh"
#include "swiglu_ops.h"

namespace swiglu {
namespace {

constexpr int kPlanSms = 152;      // grids are planned for the GB300, so that the workspace query sees no device

template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// The elements of the pack that starts at column `first` which are the row's, loaded and stored one
// by one (others are loaded as 0); `row`: column 0.
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

// The 16 bytes that start m bytes (even, below 16) into the 32 of lo and hi.
__device__ __forceinline__ uint4 shift_right(const uint4& lo, const uint4& hi, unsigned m) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
    const unsigned bits = (m & 2) * 8;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[i], w[i + 1], bits);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// How kVec columns of rows are moved: columns c .. c + kVec - 1 that start on a 16-byte boundary, c a
// multiple of kVec (kOnPacks) or any (kAligned); that start anywhere, some of them possibly before or past a
// row of kVec columns or more (kAnywhere); the same of any row, element by element (kElements); or columns
// c, c + 32, c + 64, c + 96 of fp32 rows anywhere (kSingles), which a warp's accesses take 128 bytes at a
// time.  Columns outside the row are loaded as 0 and not stored.
enum How { kOnPacks, kAligned, kAnywhere, kElements, kSingles };

// Such columns of a row, loaded and put together in two steps, so that many loads can be on their way.
// kAnywhere's, moved inside the row where they are not, come out of the three (aligned: two) aligned
// 8-byte words that hold them, each of which has at least one of them, so nothing outside the tensor's own 8-byte
// words is read.  (Out of two aligned packs, which take six more selects: the combine of 4099 tokens' 7
// rows of 1021 bf16 columns 24.5 us instead of 22.5; out of five words of 4 bytes, more loads: 21.7, but its
// gradient 26.5 instead of 24.5.)
template <class T, int HOW>
struct Cols {
    uint4 lo;
    uint2 hi;
    unsigned m;
    int moved;
    __device__ __forceinline__ void load(const T* row, int c, int D) {
        if constexpr (HOW == kOnPacks || HOW == kAligned) {
            lo = *reinterpret_cast<const uint4*>(row + c);
        } else if constexpr (HOW == kAnywhere) {
            const int inside = min(max(c, 0), D - kVec<T>);
            moved = (c - inside) * (int)sizeof(T);
            const uintptr_t at = reinterpret_cast<uintptr_t>(row + inside);
            const uint2* p = reinterpret_cast<const uint2*>(at & ~(uintptr_t)7);
            m = (unsigned)(at & 7);
            const uint2 a = p[0], b = p[1];
            lo = make_uint4(a.x, a.y, b.x, b.y);
            hi = p[m != 0 ? 2 : 1];
        } else if constexpr (HOW == kSingles) {
            static_assert(sizeof(T) == 4, "fp32 rows");
            const uint32_t* p = reinterpret_cast<const uint32_t*>(row);
            lo = make_uint4(p[c], c + 32 < D ? p[c + 32] : 0, c + 64 < D ? p[c + 64] : 0, c + 96 < D ? p[c + 96] : 0);
        } else {
            lo = load_edge(row, c, D);
        }
    }
    __device__ __forceinline__ uint4 get() const {
        if constexpr (HOW != kAnywhere) return lo;
        uint32_t w[6] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y};
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[i], w[i + 1], (m & 2) * 8);
        uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
        const uint4 none = make_uint4(0, 0, 0, 0);
        if (moved > 0) v = shift_right(v, none, moved);
        else if (moved < 0) v = shift_right(none, v, 16 + moved);
        return v;
    }
};
template <class T, int HOW>
__device__ __forceinline__ uint4 load_cols(const T* row, int c, int D) {
    Cols<T, HOW> v;
    v.load(row, c, D);
    return v.get();
}
// The same of an output, whose packs are taken on its 16-byte boundaries (first_col).
template <class T, int HOW>
__device__ __forceinline__ void store_cols(T* row, int c, int D, const uint4& v) {
    if constexpr (HOW == kSingles) {
        uint32_t* p = reinterpret_cast<uint32_t*>(row);
        p[c] = v.x;
        if (c + 32 < D) p[c + 32] = v.y;
        if (c + 64 < D) p[c + 64] = v.z;
        if (c + 96 < D) p[c + 96] = v.w;
    } else if (HOW == kElements || (HOW == kAnywhere && (c < 0 || c + kVec<T> > D))) {
        store_edge(row, c, D, v);
    } else {
        *reinterpret_cast<uint4*>(row + c) = v;
    }
}
// Item k of a row moved in singles: its first column (an item may have none).
__device__ __forceinline__ int single_col(int k) { return (k >> 5) * 128 + (k & 31); }
// First column of pack k of an output row (up to kVec - 1 before the row).
template <class T>
__device__ __forceinline__ int first_col(const T* row, int k) {
    return k * kVec<T> - (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

// Waits for what the kernels before this one in the stream wrote; the next one may come up from now on.
// (What they wrote was not constant while this kernel ran, so it is not for ld.global.nc, __ldg's.)
__device__ __forceinline__ void after_previous() {
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------- host side

// Bytes an element of `type` takes; 0 for an unknown type.
inline int type_bytes(int type) { return type == SWIGLU_FP32 ? 4 : type == SWIGLU_BF16 || type == SWIGLU_FP16 ? 2 : 0; }

inline bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// Whether `out` begins where `in` does but its rows lie elsewhere: writing it would destroy rows not yet read.
inline bool astride(const void* in, int64_t ld_in, const void* out, int64_t ld_out, int64_t rows) {
    return in == out && rows > 1 && ld_in != ld_out;
}

// f.run<T>() for the run-time type.
template <class F>
cudaError_t with_type(int type, const F& f) {
    if (type == SWIGLU_FP32) return f.template run<float>();
    if (type == SWIGLU_FP16) return f.template run<__half>();
    return f.template run<__nv_bfloat16>();
}

// A launch that may come up while the kernel before it in the stream ends: the kernel calls
// after_previous() before it reads or writes anything, and nothing is left of the launch's latency then.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// x / d for 0 <= x < 2^31 and 1 <= d < 2^31 by a product: with 2^(l - 1) < d <= 2^l and
// m = floor(2^(31 + l) / d) + 1, m d exceeds 2^(31 + l) by at most d <= 2^l, so x m / 2^(31 + l)
// exceeds x / d by less than 1 / d.
struct Divisor {
    uint32_t m, shift, d;
    static Divisor of(uint32_t d) {
        uint32_t l = 0;
        while ((uint64_t(1) << l) < d) ++l;
        return {(uint32_t)((uint64_t(1) << (31 + l)) / d + 1), 31 + l, d};
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t x) const { return (uint32_t)(((uint64_t)x * m) >> shift); }
};

}  // namespace
}  // namespace swiglu
