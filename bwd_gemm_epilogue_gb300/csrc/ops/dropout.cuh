// dropout.cuh -- the dropout of swiglu_tokens.h: which elements are kept, computed where it is used.
//
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011):
// ten rounds of two 32 x 32 -> 64 bit products on a 128-bit counter, with a 64-bit key.  One call gives
// the 16 bits of eight columns: about 60 instructions for 16 bytes of 16-bit elements, which fit beside
// their loads and stores (with 32 bits an element, a read and a write would be issue-bound).
#pragma once

#include <cmath>

#include "rows.cuh"

namespace swiglu {
namespace {

struct Dropout {
    uint64_t offset;
    const int64_t* step;       // added to offset; or null
    uint32_t key0, key1;
    uint32_t keep;             // an element's 16 bits are below it: kept
    float scale;               // 65536 / keep
};

__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint32_t h0 = __umulhi(0xD2511F53u, c0), l0 = 0xD2511F53u * c0;
        const uint32_t h1 = __umulhi(0xCD9E8D57u, c2), l1 = 0xCD9E8D57u * c2;
        c0 = h1 ^ c1 ^ k0, c1 = l1, c2 = h0 ^ c3 ^ k1, c3 = l0;
        k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ uint64_t dropout_offset(const Dropout& d) {
    return d.offset + (d.step ? (uint64_t)__ldg(reinterpret_cast<const long long*>(d.step)) : 0);
}

// The 16 bits of columns 8 b .. 8 b + 7 of a row.
__device__ __forceinline__ uint4 dropout_block(const Dropout& d, uint64_t offset, uint32_t row, uint32_t b) {
    return philox(b, row, (uint32_t)offset, (uint32_t)(offset >> 32), d.key0, d.key1);
}

// Of kVec<T> columns from c on (c >= -7; WHOLE: a multiple of kVec<T>), in order.
template <class T, bool WHOLE>
__device__ __forceinline__ uint4 dropout_bits(const Dropout& d, uint64_t offset, uint32_t row, int c) {
    const int b = c >> 3, o = c & 7;       // rounded down, where c is before the row too
    uint4 v = dropout_block(d, offset, row, (uint32_t)b);
    if constexpr (!WHOLE) {
        if (o != 0) v = shift_right(v, o + kVec<T> > 8 ? dropout_block(d, offset, row, (uint32_t)b + 1) : v, 2 * o);
    } else if constexpr (kVec<T> == 4) {
        if (o != 0) v.x = v.z, v.y = v.w;
    }
    return v;
}

// Dropped elements of a pack as 0, the others times scale.
template <class T>
__device__ __forceinline__ void drop(F2* v, const uint4& bits, uint32_t keep, float scale) {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int i = 0; i < kVec<T> / 2; ++i) {
        const float2 f = split(v[i]);
        v[i] = f2((w[i] & 0xffffu) < keep ? f.x * scale : 0.f, (w[i] >> 16) < keep ? f.y * scale : 0.f);
    }
}

// ---------------------------------------------------------------- host side

// Sets d; false where p is no probability.
inline bool dropout_of(Dropout* d, double p, uint64_t seed, uint64_t offset, const int64_t* step) {
    if (!(p >= 0.0 && p <= 1.0)) return false;
    const uint32_t keep = (uint32_t)std::nearbyint((1.0 - p) * 65536.0);
    *d = Dropout{offset, step, (uint32_t)seed, (uint32_t)(seed >> 32), keep, keep ? 65536.f / (float)keep : 0.f};
    return true;
}

}  // namespace
}  // namespace swiglu
