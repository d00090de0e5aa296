// Shared by the 8-bit block-scaled operators: element types, chunks of eight
// elements, the e4m3 conversion and the scale of a block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

namespace ap {

constexpr int kScaleBlock = 128;       // values of a row that share a scale
constexpr float kE4m3Max = 448.0f;     // largest e4m3 value
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: 1 / scale stays finite, and a block of zeros has zero codes

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}

// Two values in one 32-bit word (the lower one first).
template <typename T>
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

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Eight consecutive elements as read from memory: 16 bytes of a 16-bit type,
// 32 of float.
template <typename T>
struct Raw8 {
    uint4 w;
    __device__ __forceinline__ void unpack(float (&v)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(u[i], T());
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void unpack(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};

// The whole chunk at p, 16-byte aligned.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
        r.a = *reinterpret_cast<const float4*>(p);
        r.b = *reinterpret_cast<const float4*>(p + 4);
    } else {
        r.w = *reinterpret_cast<const uint4*>(p);
    }
    return r;
}

// The chunk at p: the first `n` of eight elements, zeros after them (n <= 0:
// nothing is read). vec: p is 16-byte aligned.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, bool vec, int64_t n) {
    if (vec && n >= 8) return load8(p);
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
        r.a = make_float4(v[0], v[1], v[2], v[3]);
        r.b = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < n ? reinterpret_cast<const uint16_t*>(p)[2 * i] : 0u;
            const uint32_t hi = 2 * i + 1 < n ? reinterpret_cast<const uint16_t*>(p)[2 * i + 1] : 0u;
            u[i] = lo | hi << 16;
        }
        r.w = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return r;
}

// Store eight values at p, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
}

// Store the first `n` of eight values. vec: p is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, int64_t n, const float (&v)[8]) {
    if (vec && n >= 8) {
        store8(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = from_f32<T>(v[i]);
}

// Store the first `n` of eight codes. vec: p is 8-byte aligned.
__device__ __forceinline__ void store_codes(uint8_t* p, bool vec, int64_t n, uint2 w) {
    if (vec && n >= 8) {
        *reinterpret_cast<uint2*>(p) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? w.x >> (8 * i) : w.y >> (8 * (i - 4))) & 0xffu);
}

// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest magnitude of three values, NaN if any is.
__device__ __forceinline__ float amax3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
    return amax3(amax3(v[0], v[1], v[2]), amax3(v[3], v[4], v[5]), amax3(v[6], v[7], 0.0f));
}

// Largest magnitudes of 16-bit values two at a time in their own type (exact:
// a maximum rounds nothing), of floats one at a time; NaN where a value is.
template <typename T>
struct Peak {  // 16-bit types: V holds two running maxima
    using V = uint32_t;
    static constexpr int kWords = 4;  // V's of a chunk of eight, for maxima by column
    static __device__ __forceinline__ V max(V a, V b) {
        V r;
        if constexpr (std::is_same_v<T, __half>)
            asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ V word(const Raw8<T>& r, int i) {
        return (i == 0 ? r.w.x : (i == 1 ? r.w.y : (i == 2 ? r.w.z : r.w.w))) & 0x7FFF7FFFu;
    }
    static __device__ __forceinline__ V chunk(const Raw8<T>& r) { return max(max(word(r, 0), word(r, 1)), max(word(r, 2), word(r, 3))); }
    static __device__ __forceinline__ float value(V v) {
        const float2 f = unpack2(v, T());
        return max_nan(f.x, f.y);
    }
    static __device__ __forceinline__ float column(const V (&v)[kWords], int i) {
        const float2 f = unpack2(v[i / 2], T());
        return i % 2 ? f.y : f.x;
    }
};
template <>
struct Peak<float> {
    using V = float;
    static constexpr int kWords = 8;
    static __device__ __forceinline__ V max(V a, V b) { return max_nan(a, b); }
    static __device__ __forceinline__ V word(const Raw8<float>& r, int i) {
        const float v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
        return fabsf(v[i]);
    }
    static __device__ __forceinline__ V chunk(const Raw8<float>& r) {
        return amax3(amax3(r.a.x, r.a.y, r.a.z), amax3(r.a.w, r.b.x, r.b.y), amax3(r.b.z, r.b.w, 0.0f));
    }
    static __device__ __forceinline__ float value(V v) { return v; }
    static __device__ __forceinline__ float column(const V (&v)[kWords], int i) { return v[i]; }
};

// A block's scale s = max(amax / 448, 2^-126) and 1 / s, both rounded to
// nearest. Every half warp of the norm and the quantiser computes them once a
// chunk, so they are written without the branches of the general operations:
// the quotient by a constant is Markstein's (the product with the rounded
// reciprocal, then one step with the exact remainder), the reciprocal one
// Newton step on the hardware's approximation. Both agree with division and
// reciprocal for every mantissa; s is never below the normal range, and an
// infinite amax, whose remainder would be NaN, has its own answer.
struct Scale {
    float s, inv;
};
__device__ __forceinline__ Scale scale_of(float amax) {
    constexpr float kRecip = 1.0f / kE4m3Max;
    const bool infinite = amax > 3.402823466e38f;
    const float q = amax * kRecip;
    const float s = max_nan(fmaf(fmaf(-kE4m3Max, q, amax), kRecip, q), kMinScale);
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    return Scale{infinite ? amax : s, infinite ? 0.0f : fmaf(y, fmaf(-s, y, 1.0f), y)};
}

// Two e4m3 codes, a in the lower byte. The magnitudes are at most 448 but for
// the rounding of the product, which the saturation absorbs; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    uint2 w;
    w.x = e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16;
    w.y = e4m3x2(v[4] * inv, v[5] * inv) | e4m3x2(v[6] * inv, v[7] * inv) << 16;
    return w;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Host: rows of `size`-byte elements that all start on `bytes`-byte boundaries.
inline bool rows_aligned(const void* p, int64_t ld, int64_t size, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * size % bytes == 0;
}

}  // namespace ap
