// convert.cuh -- element types of the operators around the block: packs of VEC elements
// moved by one load or store, and their fp32 conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace swiglu {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}

// Two 16-bit elements of a word as fp32.
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// VEC elements of T as one load moves them: 16 bytes kept as 32-bit words (the compiler would
// otherwise give each 16-bit element a register of its own), or a single element.
template <class T, int VEC>
struct Pack {
    static constexpr int kWords = 4;
    static_assert(VEC * (int)sizeof(T) == 16, "packs are 16 bytes");
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    __device__ __forceinline__ void unpack(float* o) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) {
                o[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack2<T>(w[i]);
                o[2 * i] = f.x;
                o[2 * i + 1] = f.y;
            }
        }
    }
};
template <class T>
struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void unpack(float* o) const { o[0] = to_f32(v); }
};

template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
    Pack<T, VEC> k;
    k.load(p);
    return k;
}

template <class T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const float* v) {
    if constexpr (VEC == 1) {
        *p = from_f32<T>(v[0]);
    } else {
        static_assert(VEC * (int)sizeof(T) == 16, "packs are 16 bytes");
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
            else w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ---------------------------------------------------------------- pairs of fp32

// Two fp32 values in one 64-bit register pair, for the packed fp32 instructions.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 split(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// 16 bytes of T <-> pairs.
template <class T>
__device__ __forceinline__ void unpack16(const uint4& w, F2* o) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) {
        o[0] = f2(__uint_as_float(u[0]), __uint_as_float(u[1]));
        o[1] = f2(__uint_as_float(u[2]), __uint_as_float(u[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(u[i]);
            o[i] = f2(f.x, f.y);
        }
    }
}
template <class T>
__device__ __forceinline__ uint4 pack16(const F2* v) {
    uint32_t u[4];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 f = split(v[i]);
            u[2 * i] = __float_as_uint(f.x);
            u[2 * i + 1] = __float_as_uint(f.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = split(v[i]);
            u[i] = pack2<T>(f.x, f.y);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

}  // namespace swiglu
