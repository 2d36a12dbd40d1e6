// silu(gate) * up as an MXFP8 matrix, with a checkpoint of gate and up in 8 bits, and the gradient that
// reads the checkpoint.
#include "mx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-g), within 2^-20 of it for |g| < 80: both instructions are within 2^-22, and the exponent's
// rounding adds |g| 2^-23.  (Results are rounded to four bits.)
__device__ __forceinline__ float sigmoid(float g)
{
    return rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * g));
}

// bits of the largest magnitude of the eights of four neighbouring lanes (a NaN's are the largest)
__device__ __forceinline__ uint32_t amax4(const float (&v)[8])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[i])));
    uint32_t b = __float_as_uint(m);
    b = max(b, __shfl_xor_sync(0xffffffffu, b, 1));
    return max(b, __shfl_xor_sync(0xffffffffu, b, 2));
}

// Eight u of a row of `blocks` blocks as MXFP8 (all lanes of the warp; `live` ones store).  A block's first
// lane stores its scale byte, the row's last block also the zeros behind it in its atom.
__device__ __forceinline__ void store_mx8(float (&v)[8], int rule, uint8_t* codes, uint8_t* sf, int layout,
                                          int64_t row, int u, int blocks, bool live)
{
    const uint32_t s = mx_scale_byte<E4M3>(amax4(v), rule);
    if (!live) return;
    const float scale = mx_encode_scale(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= scale;
    reinterpret_cast<uint2*>(codes)[row * (4 * blocks) + u] = s == 255u ? E4M3::zero() : E4M3::encode(v);
    if ((u & 3) == 0) {
        const int kb = u >> 2;
        if (layout == MOE_SF_CANONICAL) {
            sf[row * blocks + kb] = (uint8_t)s;
        } else {
            uint8_t* at = sf + mx_sf_tiled(0, 0, (blocks + 3) >> 2, (int)row, kb);
            at[0] = (uint8_t)s;
            if (kb == blocks - 1)
                for (int z = 1; z < 4 - (kb & 3); ++z) at[z] = 0;
        }
    }
}

// Eight u of a row of an MXFP8 matrix with canonical scales.
__device__ __forceinline__ void load_mx8(const uint8_t* codes, const uint8_t* sf, int64_t row, int u,
                                         int blocks, float (&v)[8])
{
    E4M3::decode(reinterpret_cast<const uint2*>(codes)[row * (4 * blocks) + u], v);
    const float d = mx_decode_scale(sf[row * blocks + (u >> 2)]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= d;
}

}  // namespace

// The kernels' work is 32 eights in a row's order, one a lane, which may be of several short rows.  A warp
// asks for 32 of its items at a time whether any of their rows is live, each lane for one, so that padding
// costs it one load (groups of few rows: a decode batch's rows are padding but for one in eighty).
template <typename F>
__device__ __forceinline__ void for_live_eights(const int32_t* perm_src, uint32_t n, const FastDiv& units, F work)
{
    const int lane = threadIdx.x & 31;
    const uint64_t items = ((uint64_t)n + 31) / 32, step = gridDim.x * (blockDim.x >> 5);
    for (uint64_t i0 = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i0 < items; i0 += 32 * step) {
        const uint64_t mine = i0 + lane * step;
        bool any = mine < items;
        if (any && perm_src) {
            const uint32_t last = units.div((uint32_t)min(32 * mine + 31, (uint64_t)n - 1));
            any = false;
            for (uint32_t r = units.div((uint32_t)(32 * mine)); r <= last; ++r) any = any || perm_src[r] >= 0;
        }
        for (uint32_t left = __ballot_sync(0xffffffffu, any); left; left &= left - 1) {
            const uint64_t at = 32 * (i0 + (__ffs(left) - 1) * step) + lane;
            const uint32_t i = (uint32_t)min(at, (uint64_t)n - 1), row = units.div(i);
            work((int64_t)row, (int)(i - row * units.d), at < n && !(perm_src && perm_src[row] < 0));
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) swiglu_kernel(SwigluArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int blocks = a.inter >> 5, units = a.inter >> 3;
    for_live_eights(a.perm_src, a.eights, a.units, [&](int64_t row, int u, bool live) {
        Eight<T> e = {}, f = {};
        if (live) {
            const T* x = static_cast<const T*>(a.gu) + row * a.gu_stride + 8 * u;
            e.template load<VEC>(x);
            f.template load<VEC>(x + a.inter);
        }
        float g[8], v[8];
        e.to_f32(g);
        f.to_f32(v);
        float s[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] = g[q] * sigmoid(g[q]) * v[q];
        store_mx8(s, a.rule, a.codes, a.sf, a.layout, row, u, blocks, live);
        if (a.ckpt) {
            store_mx8(g, a.rule, a.ckpt, a.ckpt_sf, MOE_SF_CANONICAL, row, u, 2 * blocks, live);
            store_mx8(v, a.rule, a.ckpt, a.ckpt_sf, MOE_SF_CANONICAL, row, u + units, 2 * blocks, live);
        }
    });
}

// With s = sigmoid(g): dg = ds u s (1 + g (1 - s)), du = ds g s.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) swiglu_back_kernel(SwigluBackArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int blocks = a.inter >> 5, units = a.inter >> 3;
    for_live_eights(a.perm_src, a.eights, a.units, [&](int64_t row, int u, bool live) {
        float g[8] = {}, v[8] = {}, d[8] = {};
        if (live) {
            Eight<T> e;
            e.template load<VEC>(static_cast<const T*>(a.ds) + row * a.ds_stride + 8 * u);
            load_mx8(a.ckpt, a.ckpt_sf, row, u, 2 * blocks, g);
            load_mx8(a.ckpt, a.ckpt_sf, row, u + units, 2 * blocks, v);
            e.to_f32(d);
        }
        float dg[8], du[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float s = sigmoid(g[q]), t = d[q] * s;
            dg[q] = t * v[q] * (1.0f + g[q] * (1.0f - s));
            du[q] = t * g[q];
        }
        if (a.dgu && live) {
            T* o = static_cast<T*>(a.dgu) + row * (int64_t)(2 * a.inter) + 8 * u;
            Eight<T> w;
            w.from_f32(dg);
            w.store(o);
            w.from_f32(du);
            w.store(o + a.inter);
        }
        if (a.codes) {
            store_mx8(dg, a.rule, a.codes, a.sf, a.layout, row, u, 2 * blocks, live);
            store_mx8(du, a.rule, a.codes, a.sf, a.layout, row, u + units, 2 * blocks, live);
        }
    });
}

SwigluKernel swiglu_kernel_for(int dtype, bool vec)
{
    switch (dtype) {
        case MOE_BF16: return vec ? swiglu_kernel<__nv_bfloat16, true> : swiglu_kernel<__nv_bfloat16, false>;
        case MOE_FP16: return vec ? swiglu_kernel<__half, true> : swiglu_kernel<__half, false>;
        default: return vec ? swiglu_kernel<float, true> : swiglu_kernel<float, false>;
    }
}

SwigluBackKernel swiglu_back_kernel_for(int dtype, bool vec)
{
    switch (dtype) {
        case MOE_BF16: return vec ? swiglu_back_kernel<__nv_bfloat16, true> : swiglu_back_kernel<__nv_bfloat16, false>;
        case MOE_FP16: return vec ? swiglu_back_kernel<__half, true> : swiglu_back_kernel<__half, false>;
        default: return vec ? swiglu_back_kernel<float, true> : swiglu_back_kernel<float, false>;
    }
}

}  // namespace moe
