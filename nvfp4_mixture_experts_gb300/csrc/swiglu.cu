// silu(gate) * up as an MXFP8 matrix, with a checkpoint of gate and up in 8 bits, and the gradient that
// reads the checkpoint.
//
// A lane has 16 columns, half of a block of 32, so that a block's scale takes one exchange and what a lane
// finds out about its row is paid for by 16 results; products and sums are of two numbers an instruction.
// 65536 rows of I 1280 bf16: forward 99 us with the checkpoint (6.0 TB/s, memory) and 72 without; the
// gradient 102 us (5.0 TB/s), bound by its instructions (0.67 of the issue slots; 250 for 8 columns of 32
// lanes; with 8 columns a lane 430, 162 us).  Held to 64 registers: four blocks an SM (74 registers, three:
// 117 us).
#include "mx.cuh"

namespace moe {

namespace {

// (numbers below 2^-126 count as 0)
__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-g), within 2^-21 + 1.25 |g| 2^-24 of itself down to g = -87 (2^-17.3 at -80), 0 below: the two
// instructions are within 2^-22 and 2^-23, the sum within 2^-24; the exponent's rounding is |g| 2^-24 and that of
// log2 e as a 32-bit number |g| 2^-26, of which a positive g's small e^-g takes little.  (MXFP8 results are rounded
// to four bits.)
__device__ __forceinline__ F2 sigmoid(F2 g)
{
    const float2 x = (g * F2(-1.4426950408889634f)).get();
    const float2 d = (F2(ex2_approx(x.x), ex2_approx(x.y)) + F2(1.0f)).get();
    return F2(rcp_approx(d.x), rcp_approx(d.y));
}

// Sixteen elements of a row, half of a block of 32; the other half is the neighbouring lane's.
constexpr int kUnit = 16, kPairs = kUnit / 2;

// bits of the block's largest magnitude (a NaN's are the largest)
__device__ __forceinline__ uint32_t amax_block(const F2 (&v)[kPairs])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) m = max_nan(m, v[i]);
    const uint32_t b = __float_as_uint(m);
    return max(b, __shfl_xor_sync(0xffffffffu, b, 1));
}

// Sixteen number `at` of an MXFP8 matrix (counted over its rows), u-th of row `row` of `blocks` blocks (all
// lanes of the warp; `live` ones store).  A block's first lane stores its scale byte, the row's last block
// also the zeros behind it in its atom.
__device__ __forceinline__ void store_mx8(const F2 (&v)[kPairs], int rule, uint8_t* codes, uint8_t* sf,
                                          int layout, uint64_t at, uint32_t row, int u, int blocks, bool live)
{
    const uint32_t s = mx_scale_byte<E4M3>(amax_block(v), rule);
    if (!live) return;
    const F2 scale(mx_encode_scale(s));
    float q[kUnit];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const float2 a = (v[i] * scale).get();
        q[2 * i] = a.x;
        q[2 * i + 1] = a.y;
    }
    uint4 c = make_uint4(f32x4_to_e4m3(q), f32x4_to_e4m3(q + 4), f32x4_to_e4m3(q + 8), f32x4_to_e4m3(q + 12));
    if (s == 255u) c = make_uint4(0u, 0u, 0u, 0u);
    reinterpret_cast<uint4*>(codes)[at] = c;
    if ((u & 1) == 0) {
        const int kb = u >> 1;
        if (layout == MOE_SF_CANONICAL) {
            sf[at >> 1] = (uint8_t)s;
        } else {
            uint8_t* to = sf + mx_sf_tiled(0, 0, (blocks + 3) >> 2, (int)row, kb);
            to[0] = (uint8_t)s;
            if (kb == blocks - 1)
                for (int z = 1; z < 4 - (kb & 3); ++z) to[z] = 0;
        }
    }
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_pairs(const T* x, F2 (&v)[kPairs])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Eight<T> e;
        e.template load<VEC>(x + 8 * h);
        float f[8];
        e.to_f32(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = F2(f[2 * i], f[2 * i + 1]);
    }
}

// The values of sixteen codes, not multiplied by their scale.
__device__ __forceinline__ void decode_pairs(uint4 c, F2 (&v)[kPairs])
{
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[4];
        e4m3x4_to_f32(w[i], f);
        v[2 * i] = F2(f[0], f[1]);
        v[2 * i + 1] = F2(f[2], f[3]);
    }
}

// The kernels' work is 32 sixteens in the rows' order, one a lane, which may be of several short rows.  A warp
// asks for 32 of its items at a time whether any of their rows is live, each lane for one, so that padding
// costs it one load (groups of few rows: a decode batch's rows are padding but for one in eighty).
template <typename F>
__device__ __forceinline__ void for_live(const int32_t* perm_src, uint32_t n, const FastDiv& units, F work)
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
            work(i, row, (int)(i - row * units.d), at < n && !(perm_src && perm_src[row] < 0));
        }
    }
}

}  // namespace

template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 4) swiglu_kernel(SwigluArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int blocks = a.inter >> 5, units = a.inter / kUnit;
    for_live(a.perm_src, a.n, a.units, [&](uint32_t i, uint32_t row, int u, bool live) {
        F2 g[kPairs], v[kPairs], s[kPairs];
#pragma unroll
        for (int q = 0; q < kPairs; ++q) g[q] = v[q] = F2(0.0f);
        if (live) {
            const T* x = static_cast<const T*>(a.gu) + row * a.gu_stride + kUnit * u;
            load_pairs<VEC>(x, g);
            load_pairs<VEC>(x + a.inter, v);
        }
#pragma unroll
        for (int q = 0; q < kPairs; ++q) s[q] = g[q] * sigmoid(g[q]) * v[q];
        store_mx8(s, a.rule, a.codes, a.sf, a.layout, i, row, u, blocks, live);
        if (a.ckpt) {
            const uint64_t at = (uint64_t)i + (uint64_t)row * units;  // sixteen u of 2 units in a row
            store_mx8(g, a.rule, a.ckpt, a.ckpt_sf, MOE_SF_CANONICAL, at, row, u, 2 * blocks, live);
            store_mx8(v, a.rule, a.ckpt, a.ckpt_sf, MOE_SF_CANONICAL, at + units, row, u + units, 2 * blocks, live);
        }
    });
}

// With s = sigmoid(g): dg = ds u s (1 + g (1 - s)), du = ds g s.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 4) swiglu_back_kernel(SwigluBackArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int blocks = a.inter >> 5, units = a.inter / kUnit;
    for_live(a.perm_src, a.n, a.units, [&](uint32_t i, uint32_t row, int u, bool live) {
        const uint64_t at = (uint64_t)i + (uint64_t)row * units;  // sixteen u of 2 units in a row
        F2 d[kPairs], g[kPairs], v[kPairs];
        uint4 cg = make_uint4(0u, 0u, 0u, 0u), cu = cg;
        uint32_t sg = 0, su = 0;
#pragma unroll
        for (int q = 0; q < kPairs; ++q) d[q] = F2(0.0f);
        if (live) {
            cg = reinterpret_cast<const uint4*>(a.ckpt)[at];
            cu = reinterpret_cast<const uint4*>(a.ckpt)[at + units];
            sg = a.ckpt_sf[at >> 1];
            su = a.ckpt_sf[(at + units) >> 1];
            load_pairs<VEC>(static_cast<const T*>(a.ds) + row * a.ds_stride + kUnit * u, d);
        }
        decode_pairs(cg, g);
        decode_pairs(cu, v);
        const F2 fg(mx_decode_scale(sg)), fu(mx_decode_scale(su));
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {   // dg in v's place, du in d's
            const F2 gq = g[q] * fg, s = sigmoid(gq), t = d[q] * s;
            const F2 rest = fma2(s, F2(-1.0f), F2(1.0f));
            v[q] = t * (v[q] * fu) * fma2(gq, rest, F2(1.0f));
            d[q] = t * gq;
        }
        if (a.dgu && live) {
            T* o = static_cast<T*>(a.dgu) + kUnit * at;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                float f[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 p = (h < 2 ? v[4 * h + q] : d[4 * (h - 2) + q]).get();
                    f[2 * q] = p.x;
                    f[2 * q + 1] = p.y;
                }
                Eight<T> w;
                w.from_f32(f);
                w.store(o + (h < 2 ? 8 * h : a.inter + 8 * (h - 2)));
            }
        }
        if (a.codes) {
            store_mx8(v, a.rule, a.codes, a.sf, a.layout, at, row, u, 2 * blocks, live);
            store_mx8(d, a.rule, a.codes, a.sf, a.layout, at + units, row, u + units, 2 * blocks, live);
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
