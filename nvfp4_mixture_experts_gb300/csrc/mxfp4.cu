// MXFP4: quantisation (of a matrix or of its transpose) and the tiled scale layout.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float elem_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float elem_f32(float v) { return v; }
__device__ __forceinline__ void set_elem(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void set_elem(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void set_elem(float& d, float v) { d = v; }

// The scale byte of a block from the bits of its largest magnitude (the magnitudes' bits are
// ordered as the magnitudes are, infinities and NaNs above every number): exponent field - 2, one
// more under the ceil rule when the significand passes 1.5 (m = 1.5 * 2^(e+2) is 6 * 2^e), at
// least 0 (2^-127).  255 for an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits, int rule)
{
    if (amax_bits >= 0x7F800000u) return 255u;
    int b = (int)(amax_bits >> 23) - 2;
    if (rule == MOE_MX_CEIL && (amax_bits & 0x7FFFFFu) > 0x400000u) ++b;
    return (uint32_t)max(b, 0);
}

// 2^(127 - s): what elements of a block with scale byte s (0..253) are multiplied by.
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

// Stores the scale byte of block kb of row r; the last block of a row also zeroes the scales of
// the blocks past it in its atom.
__device__ __forceinline__ void store_scale(uint8_t* sf, int layout, int64_t b, int R, int r,
                                            int blocks, int kb, uint32_t s)
{
    if (layout == MOE_SF_CANONICAL) {
        sf[(b * R + r) * blocks + kb] = (uint8_t)s;
        return;
    }
    const size_t o = mx_sf_tiled(b, (R + 127) >> 7, (blocks + 3) >> 2, r, kb);
    sf[o] = (uint8_t)s;
    if (kb == blocks - 1)
        for (int i = (kb & 3) + 1; i < 4; ++i) sf[o - (kb & 3) + i] = 0;
}

}  // namespace

// ------------------------------------------------------------------ a matrix

// Eight elements per thread, four neighbouring threads per block of 32.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_quant_kernel(MxQuantArgs a)
{
    const int units = a.cols >> 3;  // eights per row: a multiple of 4, so a block's four threads
                                    // are in one row and one warp
    const int64_t n = (int64_t)a.batch * a.rows * units;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const int64_t n_round = (n + 31) / 32 * 32;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_round; i += step) {
        const bool in = i < n;
        const int64_t row = in ? i / units : 0;
        const int u = (int)(in ? i % units : 0);
        const int64_t b = row / a.rows;
        const int r = (int)(row % a.rows);
        const bool live = in && !(a.perm_src && a.perm_src[r] < 0);
        float v[8] = {};
        if (live) {
            const T* x = static_cast<const T*>(a.x) + b * a.batch_stride + r * a.row_stride + u * 8;
            if constexpr (VEC) {
                constexpr int kPer = 16 / (int)sizeof(T);
                alignas(16) T e[8];
#pragma unroll
                for (int q = 0; q < 8 / kPer; ++q)
                    reinterpret_cast<uint4*>(e)[q] = reinterpret_cast<const uint4*>(x)[q];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = elem_f32(e[q]);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = elem_f32(x[q]);
            }
        }
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (!live) continue;
        const uint32_t s = mx_scale_byte(m, a.rule);
        uint32_t codes = 0;
        if (s != 255u) {
            const float scale = mx_encode_scale(s);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= scale;
            codes = f32x8_to_e2m1(v);
        }
        reinterpret_cast<uint32_t*>(a.codes)[i] = codes;
        if ((u & 3) == 0) store_scale(a.sf, a.layout, b, a.rows, r, units >> 2, u >> 2, s);
        if (a.values) {
            const float d = mx_decode_scale(s);
            e2m1x8_to_f32(codes, v);
            alignas(16) T e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) set_elem(e[q], v[q] * d);
            T* o = static_cast<T*>(a.values) + i * 8;
#pragma unroll
            for (int q = 0; q < (int)sizeof(T) / 2; ++q)
                reinterpret_cast<uint4*>(o)[q] = reinterpret_cast<const uint4*>(e)[q];
        }
    }
}

MxQuantKernel mx_quant_kernel_for(int dtype, bool vec)
{
    switch (dtype) {
        case MOE_BF16: return vec ? mx_quant_kernel<__nv_bfloat16, true> : mx_quant_kernel<__nv_bfloat16, false>;
        case MOE_FP16: return vec ? mx_quant_kernel<__half, true> : mx_quant_kernel<__half, false>;
        default: return vec ? mx_quant_kernel<float, true> : mx_quant_kernel<float, false>;
    }
}

// ------------------------------------------------------------------ a matrix's transpose

// A thread per (column, 32 rows): the block of 32 of the transposed row is the thread's own.
template <typename T>
__global__ void __launch_bounds__(128) mx_quant_transposed_kernel(MxQuantArgs a)
{
    const int blocks = a.rows >> 5;
    const int64_t n = (int64_t)a.batch * blocks * a.cols;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        const int c = (int)(i % a.cols);
        const int kb = (int)(i / a.cols % blocks);
        const int64_t b = i / a.cols / blocks;
        const T* x = static_cast<const T*>(a.x) + b * a.batch_stride +
                     (int64_t)kb * 32 * a.row_stride + c;
        float v[32];
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 32; ++q) {
            v[q] = elem_f32(x[q * a.row_stride]);
            m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
        }
        const uint32_t s = mx_scale_byte(m, a.rule);
        uint32_t codes[4] = {};
        if (s != 255u) {
            const float scale = mx_encode_scale(s);
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] *= scale;
#pragma unroll
            for (int q = 0; q < 4; ++q) codes[q] = f32x8_to_e2m1(v + 8 * q);
        }
        const int64_t o = ((b * a.cols + c) * blocks + kb) * 32;
        *reinterpret_cast<uint4*>(a.codes + o / 2) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
        store_scale(a.sf, a.layout, b, a.cols, c, blocks, kb, s);
        if (a.values) {
            const float d = mx_decode_scale(s);
            alignas(16) T e[32];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float f[8];
                e2m1x8_to_f32(codes[q], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) set_elem(e[8 * q + j], f[j] * d);
            }
            uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(a.values) + o);
#pragma unroll
            for (int q = 0; q < 2 * (int)sizeof(T); ++q) to[q] = reinterpret_cast<const uint4*>(e)[q];
        }
    }
}

MxQuantKernel mx_quant_transposed_kernel_for(int dtype)
{
    switch (dtype) {
        case MOE_BF16: return mx_quant_transposed_kernel<__nv_bfloat16>;
        case MOE_FP16: return mx_quant_transposed_kernel<__half>;
        default: return mx_quant_transposed_kernel<float>;
    }
}

// ------------------------------------------------------------------ scale layout

// A thread per 4-byte word of the tiled layout: four scales of one row.
__global__ void __launch_bounds__(256) mx_tile_scales_kernel(const uint8_t* sf, int batch, int rows,
                                                             int blocks, uint8_t* tiled)
{
    const int RB = (rows + 127) >> 7, KA = (blocks + 3) >> 2;
    const int64_t n = (int64_t)batch * RB * KA * 128;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int w = (int)(i & 127);                 // word of the atom: row (w % 4) * 32 + w / 4
        const int64_t atom = i >> 7;
        const int ka = (int)(atom % KA);
        const int64_t rb = atom / KA;
        const int r = (int)(rb % RB) * 128 + (w & 3) * 32 + (w >> 2);
        const int64_t b = rb / RB;
        uint32_t word = 0;
        if (r < rows)
            for (int kk = 0; kk < 4; ++kk)
                if (ka * 4 + kk < blocks)
                    word |= (uint32_t)sf[(b * rows + r) * blocks + ka * 4 + kk] << (8 * kk);
        reinterpret_cast<uint32_t*>(tiled)[i] = word;
    }
}

}  // namespace moe
