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

// Stores the scale bytes of blocks kb .. kb + 3 of row r (kb a multiple of 4; the bytes of blocks
// past the row's end are zero, as the tiled layout wants them).
__device__ __forceinline__ void store_scales(uint8_t* sf, int layout, int64_t b, int R, int r,
                                             int blocks, int kb, uint32_t word)
{
    if (layout == MOE_SF_TILED) {
        *reinterpret_cast<uint32_t*>(sf + mx_sf_tiled(b, (R + 127) >> 7, (blocks + 3) >> 2, r, kb)) = word;
    } else {
        uint8_t* o = sf + (b * R + r) * blocks + kb;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (kb + i < blocks) o[i] = (uint8_t)(word >> (8 * i));
    }
}

}  // namespace

// ------------------------------------------------------------------ a matrix

// Eight elements per thread, four neighbouring threads per block of 32: a warp's codes are 128
// contiguous bytes.  A warp takes a run of kMxQuantRun eights of a row, its loads in flight
// together.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_quant_kernel(MxQuantArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kPer = kMxQuantRun / 32;
    const int lane = threadIdx.x & 31;
    const int units = a.cols >> 3;  // eights per row, a multiple of 4
    const int runs = (units + kMxQuantRun - 1) / kMxQuantRun;
    const int64_t items = (int64_t)a.batch * a.rows * runs;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < items; i += step) {
        const int64_t row = i / runs;
        const int u0 = (int)(i - row * runs) * kMxQuantRun + lane;
        const int64_t b = a.batch == 1 ? 0 : row / a.rows;
        const int r = (int)(row - b * a.rows);
        if (a.perm_src && a.perm_src[r] < 0) continue;
        const T* x = static_cast<const T*>(a.x) + b * a.batch_stride + r * a.row_stride;
        alignas(16) T e[kPer][8];
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int u = u0 + 32 * p;
            if (u < units) {
                if constexpr (VEC) {
#pragma unroll
                    for (int q = 0; q < (int)sizeof(T) / 2; ++q)
                        reinterpret_cast<uint4*>(e[p])[q] = reinterpret_cast<const uint4*>(x + (int64_t)u * 8)[q];
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) e[p][q] = x[(int64_t)u * 8 + q];
                }
            }
        }
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const int u = u0 + 32 * p;
            if (u - lane >= units) break;
            const bool in = u < units;
            float v[8];
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                v[q] = in ? elem_f32(e[p][q]) : 0.0f;
                m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
            }
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t s = mx_scale_byte(m, a.rule);
            // the scales of four blocks (16 lanes) in one word
            uint32_t word = in ? s << (8 * ((lane >> 2) & 3)) : 0u;
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            word |= __shfl_xor_sync(0xffffffffu, word, 8);
            if (!in) continue;
            uint32_t codes = 0;
            if (s != 255u) {
                const float scale = mx_encode_scale(s);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= scale;
                codes = f32x8_to_e2m1(v);
            }
            const int64_t at = row * units + u;
            reinterpret_cast<uint32_t*>(a.codes)[at] = codes;
            if ((lane & 15) == 0) store_scales(a.sf, a.layout, b, a.rows, r, units >> 2, u >> 2, word);
            if (a.values) {
                const float d = mx_decode_scale(s);
                e2m1x8_to_f32(codes, v);
                alignas(16) T o[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) set_elem(o[q], v[q] * d);
#pragma unroll
                for (int q = 0; q < (int)sizeof(T) / 2; ++q)
                    reinterpret_cast<uint4*>(static_cast<T*>(a.values) + at * 8)[q] =
                        reinterpret_cast<const uint4*>(o)[q];
            }
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

// A block of threads per tile of 128 rows x 64 columns, a thread per (column, 32 rows), whose
// block of 32 of the transposed row is its own: the loads run along the rows of x (lanes =
// columns).  The transposed rows go out through shared memory, 128 elements (64 code bytes) of a
// row at a time; a row's four scale bytes are one word.
template <typename T>
__global__ void __launch_bounds__(256) mx_quant_transposed_kernel(MxQuantArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kCols = 64;
    constexpr int kPitch = 128 + 16 / (int)sizeof(T);  // elements; 16-byte accesses of neighbouring
                                                       // columns fall into different banks
    __shared__ alignas(16) T s_val[kCols * kPitch];
    __shared__ uint4 s_code[kCols][5];                 // 64 bytes and 16 of padding per column
    __shared__ uint32_t s_scale[kCols];
    const int rt = (a.rows + 127) >> 7, ct = (a.cols + kCols - 1) / kCols;
    const int blocks = a.rows >> 5;
    const int c = threadIdx.x % kCols, rq = threadIdx.x / kCols;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tiles = (int64_t)a.batch * rt * ct;
    for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x) {
        const int64_t b = i / ((int64_t)rt * ct);
        const int t = (int)(i - b * rt * ct);
        const int tr = t / ct, c0 = (t - tr * ct) * kCols, kb = tr * 4 + rq;
        const int R = min(128, a.rows - tr * 128), C = min(kCols, a.cols - c0);  // this tile's
        const bool in = c < C && kb < blocks;
        if (threadIdx.x < kCols) s_scale[threadIdx.x] = 0;
        __syncthreads();
        if (in) {
            const T* x = static_cast<const T*>(a.x) + b * a.batch_stride +
                         (int64_t)kb * 32 * a.row_stride + c0 + c;
            T e[32];
#pragma unroll
            for (int q = 0; q < 32; ++q) e[q] = x[q * a.row_stride];
            float v[32];
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                v[q] = elem_f32(e[q]);
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
            s_code[c][rq] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            reinterpret_cast<uint8_t*>(&s_scale[c])[rq] = (uint8_t)s;
            if (a.values) {
                const float d = mx_decode_scale(s);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float f[8];
                    e2m1x8_to_f32(codes[q], f);
                    alignas(16) T o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) set_elem(o[j], f[j] * d);
                    uint4* to = reinterpret_cast<uint4*>(&s_val[c * kPitch + rq * 32 + 8 * q]);
#pragma unroll
                    for (int j = 0; j < (int)sizeof(T) / 2; ++j) to[j] = reinterpret_cast<const uint4*>(o)[j];
                }
            }
        }
        __syncthreads();
        const int64_t row0 = (b * a.cols + c0) * a.rows + tr * 128;  // element of column c0's row
        if (threadIdx.x < C)
            store_scales(a.sf, a.layout, b, a.cols, c0 + threadIdx.x, blocks, tr * 4, s_scale[threadIdx.x]);
        // codes: a thread per 16 bytes, four per column
        if (threadIdx.x / 4 < C && (threadIdx.x & 3) * 32 < R)
            *reinterpret_cast<uint4*>(a.codes + (row0 + (int64_t)(threadIdx.x >> 2) * a.rows) / 2 +
                                      (threadIdx.x & 3) * 16) = s_code[threadIdx.x >> 2][threadIdx.x & 3];
        if (a.values) {
            constexpr int kEl = 16 / (int)sizeof(T), kLanes = 128 / kEl;  // lanes per column
            for (int q = warp * (32 / kLanes) + lane / kLanes; q < C; q += 8 * (32 / kLanes)) {
                const int e0 = (lane % kLanes) * kEl;
                if (e0 < R)
                    *reinterpret_cast<uint4*>(static_cast<T*>(a.values) + row0 + (int64_t)q * a.rows + e0) =
                        *reinterpret_cast<const uint4*>(&s_val[q * kPitch + e0]);
            }
        }
        __syncthreads();
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
