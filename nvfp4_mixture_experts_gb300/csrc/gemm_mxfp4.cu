// The grouped MXFP4 product: out[r][n] = sum_i A[r][i] W_g[n][i] over the rows r of each group g.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float e2m1_f32(uint32_t c)
{
    const uint32_t m = c & 7u;
    const float v = m < 2 ? 0.5f * (float)m : (float)(2 + (m & 1)) * (float)(1 << (m >> 1)) * 0.25f;
    return (c & 8u) ? -v : v;
}

__device__ __forceinline__ float mx_scale(uint32_t s)
{
    return s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s == 0 ? 0x400000u : s << 23);
}

__device__ __forceinline__ void store_out(float v, __nv_bfloat16* o) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_out(float v, __half* o) { *o = __float2half_rn(v); }
__device__ __forceinline__ void store_out(float v, float* o) { *o = v; }

}  // namespace

// A block per (32 rows of a group, 64 columns), 32 contraction elements at a time decoded into
// shared memory; a thread sums 8 outputs.
template <typename T>
__global__ void __launch_bounds__(256) mx_gemm_kernel(MxGemmArgs a)
{
    __shared__ float sA[32][33], sW[64][33];
    const int n0 = blockIdx.x * 64, KA = ((a.K >> 5) + 3) >> 2, NB = (a.N + 127) >> 7;
    for (int64_t r0 = (int64_t)blockIdx.y * 32; r0 < a.rows_cap; r0 += (int64_t)gridDim.y * 32) {
        int g = 0;
        int64_t end = a.rows_cap;
        if (a.offsets) {
            int lo = 0, hi = a.G - 1;  // the last group that starts at or before r0
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.offsets[mid] <= r0) lo = mid;
                else hi = mid - 1;
            }
            g = lo;
            const int64_t first = a.offsets[g], cnt = a.counts[g];
            end = first + cnt;
            if (cnt > 0 && (first < 0 || (first & 127) || end > a.rows_cap)) {
                if (threadIdx.x == 0) set_status(a.status, MOE_DEV_BAD_INDEX);
                continue;
            }
            if (r0 < first || r0 >= end) continue;
        }
        const int m = threadIdx.x & 31, nq = threadIdx.x >> 5;
        float acc[8] = {};
        for (int kb = 0; kb < a.K / 32; ++kb) {
            for (int i = threadIdx.x; i < 96 * 16; i += 256) {
                const int row = i >> 4, byte = i & 15;
                uint32_t c = 0;
                float s = 0.0f;
                if (row < 32) {
                    if (r0 + row < end) {
                        c = a.a_codes[(r0 + row) * (a.K / 2) + kb * 16 + byte];
                        s = mx_scale(a.a_sf[mx_sf_tiled(0, 0, KA, (int)(r0 + row), kb)]);
                    }
                } else if (n0 + row - 32 < a.N) {
                    const int n = n0 + row - 32;
                    c = a.w_codes[((int64_t)g * a.N + n) * (a.K / 2) + kb * 16 + byte];
                    s = mx_scale(a.w_sf[mx_sf_tiled(g, NB, KA, n, kb)]);
                }
                float* d = row < 32 ? sA[row] : sW[row - 32];
                d[2 * byte] = e2m1_f32(c & 15u) * s;
                d[2 * byte + 1] = e2m1_f32(c >> 4) * s;
            }
            __syncthreads();
            for (int i = 0; i < 32; ++i) {
                const float x = sA[m][i];
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = fmaf(x, sW[nq * 8 + q][i], acc[q]);
            }
            __syncthreads();
        }
        if (r0 + m < end)
            for (int q = 0; q < 8; ++q)
                if (n0 + nq * 8 + q < a.N)
                    store_out(acc[q], static_cast<T*>(a.out) + (r0 + m) * a.out_stride + n0 + nq * 8 + q);
    }
}

MxGemmKernel mx_gemm_kernel_for(int out_dtype)
{
    switch (out_dtype) {
        case MOE_BF16: return mx_gemm_kernel<__nv_bfloat16>;
        case MOE_FP16: return mx_gemm_kernel<__half>;
        default: return mx_gemm_kernel<float>;
    }
}

}  // namespace moe
