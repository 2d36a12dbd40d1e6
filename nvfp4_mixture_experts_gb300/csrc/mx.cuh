// Device helpers of the kernels that write or read MX block formats: eight elements of a row in
// registers, the power-of-two scale of 32 elements, and the E2M1 and E4M3 conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.cuh"

namespace moe {

// Two fp32 numbers, multiplied and added in one instruction.
struct F2 {
    uint64_t v;
    F2() = default;
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
    __device__ __forceinline__ float2 get() const
    {
        float2 r;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
        return r;
    }
    __device__ __forceinline__ F2 operator*(F2 o) const
    {
        F2 r;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(v), "l"(o.v));
        return r;
    }
    __device__ __forceinline__ F2 operator+(F2 o) const
    {
        F2 r;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(v), "l"(o.v));
        return r;
    }
};
// a b + c
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Eight elements of a row as raw words.
template <typename T>
struct Eight {
    static constexpr int kWords = 2 * (int)sizeof(T);
    uint32_t w[kWords];

    template <bool VEC>
    __device__ __forceinline__ void load(const T* x)
    {
        if constexpr (VEC) {
#pragma unroll
            for (int q = 0; q < kWords / 4; ++q) {
                const uint4 v = reinterpret_cast<const uint4*>(x)[q];
                w[4 * q] = v.x;
                w[4 * q + 1] = v.y;
                w[4 * q + 2] = v.z;
                w[4 * q + 3] = v.w;
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = reinterpret_cast<const uint32_t*>(x)[q];
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = h[2 * q] | (uint32_t)h[2 * q + 1] << 16;
        }
    }
    // the first n of the eight, zeros behind them
    __device__ __forceinline__ void load_some(const T* x, int n)
    {
#pragma unroll
        for (int q = 0; q < kWords; ++q) w[q] = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < n) w[q] = reinterpret_cast<const uint32_t*>(x)[q];
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < n) w[q / 2] |= (uint32_t)h[q] << (16 * (q & 1));
        }
    }
    // bits (as fp32) of the largest magnitude over the eights of four neighbouring lanes; 16-bit
    // types compare two magnitudes at a time (their bits are ordered as they are)
    __device__ __forceinline__ uint32_t amax4() const
    {
        uint32_t m = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int q = 0; q < 8; ++q) m = max(m, w[q] & 0x7FFFFFFFu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) m = max_u16x2(m, w[q] & 0x7FFF7FFFu);
            m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
            return bits16_f32(max(m & 0xFFFFu, m >> 16));
        }
    }
    // the bits, as fp32, of a 16-bit element's value
    static __device__ __forceinline__ uint32_t bits16_f32(uint32_t h)
    {
        if constexpr (std::is_same<T, __half>::value)
            return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
        else return h << 16;
    }
    __device__ __forceinline__ void to_f32(float (&v)[8]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(w[q]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (std::is_same<T, __half>::value) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[q]));
                    v[2 * q] = f.x;
                    v[2 * q + 1] = f.y;
                } else {
                    v[2 * q] = __uint_as_float(w[q] << 16);
                    v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
                }
            }
        }
    }
    __device__ __forceinline__ void from_f32(const float (&v)[8])
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(v[q]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (std::is_same<T, __half>::value) {
                    const __half2 h = __floats2half2_rn(v[2 * q], v[2 * q + 1]);
                    w[q] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
                    w[q] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        }
    }
    __device__ __forceinline__ void store(T* x) const  // 16-byte aligned
    {
#pragma unroll
        for (int q = 0; q < kWords / 4; ++q)
            reinterpret_cast<uint4*>(x)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
    // the first n of the eight, an element at a time
    __device__ __forceinline__ void store_some(T* x, int n) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < n) reinterpret_cast<uint32_t*>(x)[q] = w[q];
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < n) reinterpret_cast<uint16_t*>(x)[q] = (uint16_t)(w[q / 2] >> (16 * (q & 1)));
        }
    }
    static __device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};

// The largest of m and the magnitudes of a pair (NaN, where one is).
__device__ __forceinline__ float max_nan(float m, F2 p)
{
    const float2 v = p.get();
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v.x), "f"(v.y));
    return m;
}

template <typename T>
__device__ __forceinline__ void to_pairs(const Eight<T>& e, F2 (&v)[4])
{
    float f[8];
    e.to_f32(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = F2(f[2 * i], f[2 * i + 1]);
}

template <typename T>
__device__ __forceinline__ void from_pairs(const F2 (&v)[4], Eight<T>& e)
{
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = v[i].get();
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
    e.from_f32(f);
}

// 2^(127 - s): what elements of a block with scale byte s (0..253) are multiplied by (255: any
// number; its codes are not used).
__device__ __forceinline__ float mx_encode_scale(uint32_t s)
{
    return __uint_as_float((254u - s) << 23);
}

// 2^(s - 127); s = 255: NaN.
__device__ __forceinline__ float mx_decode_scale(uint32_t s)
{
    return s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s == 0 ? 0x400000u : s << 23);
}

// The values of eight E2M1 codes (a 32-bit word, the first in the lowest nibble).
__device__ __forceinline__ void e2m1x8_to_f32(uint32_t codes, float (&v)[8])
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = *reinterpret_cast<const __half2*>(&h[i]);
        v[2 * i] = __low2float(p);
        v[2 * i + 1] = __high2float(p);
    }
}

// Four fp32 values -> four E4M3 codes (round to nearest even, saturating at +-448), the first in the
// lowest byte.
__device__ __forceinline__ uint32_t f32x4_to_e4m3(const float* v)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
    return lo | (uint32_t)hi << 16;
}

// The values of four E4M3 codes.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float* v)
{
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(c & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(c >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

// The element formats.  kTop: the exponent of the format's largest power of two; kHalf: the significand
// bits (fp32) above which a magnitude of that exponent passes the format's largest number, 1.5 * 2^2
// or 1.75 * 2^8; Codes: eight codes.
struct E2M1 {
    static constexpr int kTop = 2;
    static constexpr uint32_t kHalf = 0x400000u;
    using Codes = uint32_t;
    static __device__ __forceinline__ Codes encode(const float (&v)[8]) { return f32x8_to_e2m1(v); }
    static __device__ __forceinline__ Codes zero() { return 0u; }
    static __device__ __forceinline__ void decode(Codes c, float (&v)[8]) { e2m1x8_to_f32(c, v); }
};
struct E4M3 {
    static constexpr int kTop = 8;
    static constexpr uint32_t kHalf = 0x600000u;
    using Codes = uint2;
    static __device__ __forceinline__ Codes encode(const float (&v)[8])
    {
        return make_uint2(f32x4_to_e4m3(v), f32x4_to_e4m3(v + 4));
    }
    static __device__ __forceinline__ Codes zero() { return make_uint2(0u, 0u); }
    static __device__ __forceinline__ void decode(Codes c, float (&v)[8])
    {
        e4m3x4_to_f32(c.x, v);
        e4m3x4_to_f32(c.y, v + 4);
    }
};

// The scale byte of a block from the bits of its largest magnitude (the magnitudes' bits are
// ordered as the magnitudes are, infinities and NaNs above every number): exponent field - kTop, one
// more under the ceil rule when the significand passes the format's largest (1.5 * 2^(e+2) is 6 * 2^e,
// 1.75 * 2^(e+8) is 448 * 2^e), at least 0 (2^-127).  255 for an infinity or a NaN.
template <typename F>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits, int rule)
{
    if (amax_bits >= 0x7F800000u) return 255u;
    int b = (int)(amax_bits >> 23) - F::kTop;
    if (rule == MOE_MX_CEIL && (amax_bits & 0x7FFFFFu) > F::kHalf) ++b;
    return (uint32_t)max(b, 0);
}

}  // namespace moe
