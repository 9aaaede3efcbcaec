// dropout.cuh -- the dropout of swiglu_tokens.h: which elements are kept, computed where it is used.
//
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011):
// ten rounds of two 32 x 32 -> 64 bit products on a 128-bit counter, with a 64-bit key.  One call gives
// the 16 bits of eight columns: 40 instructions for 16 bytes of 16-bit elements, which fit beside their
// loads and stores (32 bits an element would take twice as many).
#pragma once

#include <cmath>

#include "rows.cuh"

namespace swiglu {
namespace {

struct Dropout {
    uint64_t offset;
    const int64_t* step;       // added to offset; or null
    uint32_t keys[20];         // two for each round
    uint32_t keep;             // an element's 16 bits are below it: kept
    float scale;               // 65536 / keep
};

// The rounds' keys come from the kernel's parameters, so a round is two products and two three-way xors.
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, const uint32_t* keys) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ keys[2 * i], c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ keys[2 * i + 1], c3 = (uint32_t)p0;
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ uint64_t dropout_offset(const Dropout& d) {
    return d.offset + (d.step ? (uint64_t)*d.step : 0);
}

// The 16 bits of columns 8 b .. 8 b + 7 of a row.
__device__ __forceinline__ uint4 dropout_block(const Dropout& d, uint64_t offset, uint32_t row, uint32_t b) {
    return philox(b, row, (uint32_t)offset, (uint32_t)(offset >> 32), d.keys);
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

// A bit for each of columns 8 b .. 8 b + 7: whether it is kept.
__device__ __forceinline__ uint8_t dropout_byte(const Dropout& d, uint64_t offset, uint32_t row, uint32_t b) {
    const uint4 v = dropout_block(d, offset, row, b);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bits |= ((w[i] & 0xffffu) < d.keep ? 1u : 0u) << 2 * i | ((w[i] >> 16) < d.keep ? 2u : 0u) << 2 * i;
    return (uint8_t)bits;
}
template <class T>
__device__ __forceinline__ void drop(F2* v, uint32_t bits, float scale) {
#pragma unroll
    for (int i = 0; i < kVec<T> / 2; ++i) {
        const float2 f = split(v[i]);
        v[i] = f2(bits & 1u << 2 * i ? f.x * scale : 0.f, bits & 2u << 2 * i ? f.y * scale : 0.f);
    }
}

// ---------------------------------------------------------------- host side

// Sets d; false where p is no probability.
inline bool dropout_of(Dropout* d, double p, uint64_t seed, uint64_t offset, const int64_t* step) {
    if (!(p >= 0.0 && p <= 1.0)) return false;
    const uint32_t keep = (uint32_t)std::nearbyint((1.0 - p) * 65536.0);
    d->offset = offset, d->step = step, d->keep = keep, d->scale = keep ? 65536.f / (float)keep : 0.f;
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    for (int i = 0; i < 10; ++i, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) d->keys[2 * i] = k0, d->keys[2 * i + 1] = k1;
    return true;
}

}  // namespace
}  // namespace swiglu
