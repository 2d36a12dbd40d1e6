// Root-mean-square norm with the residual's addition, its result in the rows' own type and as an MXFP8
// matrix, and its gradient.
#include "mx.cuh"

namespace moe {

namespace {

// Sums of a row's threads: a warp's (ONE) or, through shared memory, a block's.  buf alternates from row
// to row, so that a row's sums are not written while another's are read.
template <bool ONE>
__device__ __forceinline__ float row_sum(float v, float (*s_part)[32], int buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (!ONE) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) s_part[buf][warp] = v;
        __syncthreads();
        v = lane < (int)(blockDim.x >> 5) ? s_part[buf][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// Eight u of a row of H elements.
template <bool VEC, typename T>
__device__ __forceinline__ void load_eight(Eight<T>& e, const T* row, int u, int H)
{
    if constexpr (VEC) e.template load<true>(row + 8 * u);
    else e.load_some(row + 8 * u, H - 8 * u);
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_eight(const Eight<T>& e, T* row, int u, int H)
{
    if constexpr (VEC) e.store(row + 8 * u);
    else e.store_some(row + 8 * u, H - 8 * u);
}

}  // namespace

// A row in the registers of one warp (ONE, eight rows a block) or of one block, PER eights a thread: each
// input is read once and each output written once.
template <typename T, int PER, bool ONE, bool VEC>
__global__ void __launch_bounds__(ONE ? 256 : 1024) norm_kernel(NormArgs a)
{
    __shared__ float s_part[2][32];
    pdl_wait();
    pdl_trigger();
    const int tid = ONE ? threadIdx.x & 31 : threadIdx.x, nt = ONE ? 32 : blockDim.x;
    const int lane = threadIdx.x & 31;
    const int units = div_up(a.H, 8), blocks = a.H >> 5, KA = (blocks + 3) >> 2;
    const int step = ONE ? gridDim.x * 8 : gridDim.x;
    int buf = 0;
    for (int64_t row = ONE ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x; row < a.T; row += step) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        Eight<T> e[PER] = {}, r[PER] = {};
#pragma unroll
        for (int p = 0; p < PER; ++p)
            if (tid + p * nt < units) {
                load_eight<VEC>(e[p], x, tid + p * nt, a.H);
                if (a.res)
                    load_eight<VEC>(r[p], static_cast<const T*>(a.res) + row * a.res_stride, tid + p * nt, a.H);
            }
        float v[PER][8], sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            e[p].to_f32(v[p]);
            if (a.res) {
                float q[8];
                r[p].to_f32(q);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[p][i] += q[i];
                // the stream holds h in its own type, and its norm is that of what it holds
                e[p].from_f32(v[p]);
                e[p].to_f32(v[p]);
                if (a.h && tid + p * nt < units)
                    store_eight<VEC>(e[p], static_cast<T*>(a.h) + row * a.h_stride, tid + p * nt, a.H);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(v[p][i], v[p][i], sum);
        }
        sum = row_sum<ONE>(sum, s_part, buf);
        buf ^= 1;
        const float rstd = rsqrtf(sum / (float)a.H + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int u = tid + p * nt;
            const bool in = u < units;
            if (u - lane >= units) break;  // (a warp's lanes stay together)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] *= rstd;
            if (a.w) {
                Eight<T> w = {};
                if (in) load_eight<VEC>(w, static_cast<const T*>(a.w), u, a.H);
                float q[8];
                w.to_f32(q);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[p][i] *= q[i];
            }
            if (a.y && in) {
                Eight<T> o;
                o.from_f32(v[p]);
                store_eight<VEC>(o, static_cast<T*>(a.y) + row * a.y_stride, u, a.H);
            }
            if (a.codes) {  // H % 32 == 0: a block's four lanes are in or out together
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[p][i]) & 0x7FFFFFFFu);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t s = mx_scale_byte<E4M3>(m, a.rule);
                // the scales of four blocks (16 lanes) in one word, zero past the row's end
                uint32_t word = in ? s << (8 * ((lane >> 2) & 3)) : 0u;
                word |= __shfl_xor_sync(0xffffffffu, word, 4);
                word |= __shfl_xor_sync(0xffffffffu, word, 8);
                if (!in) continue;
                const float scale = mx_encode_scale(s);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[p][i] *= scale;
                reinterpret_cast<uint2*>(a.codes)[row * units + u] = s == 255u ? E4M3::zero() : E4M3::encode(v[p]);
                const int kb = u >> 2;
                if (a.layout == MOE_SF_TILED) {
                    if ((lane & 15) == 0)
                        *reinterpret_cast<uint32_t*>(a.sf + mx_sf_tiled(0, 0, KA, (int)row, kb)) = word;
                } else if ((lane & 3) == 0) {
                    a.sf[row * blocks + kb] = (uint8_t)s;
                }
            }
        }
    }
}

// With d = dy w and x^ = h rstd: dx = rstd (d - x^ mean(d x^)) + dh, dw = sum over the rows of dy x^.  A
// block (ONE: a warp) takes every (number of parts)-th row and holds its part of dw in registers; the
// parts are added up in order by the second kernel, so results do not change from call to call.
template <typename T, int PER, bool ONE, bool VEC, int NT>
__global__ void __launch_bounds__(NT) norm_back_kernel(NormBackArgs a)
{
    __shared__ float s_part[2][32];
    pdl_wait();
    pdl_trigger();
    const int tid = ONE ? threadIdx.x & 31 : threadIdx.x, nt = ONE ? 32 : blockDim.x;
    const int units = div_up(a.H, 8);
    const int part = ONE ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    float acc[PER][8] = {}, w[PER][8];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        Eight<T> e = {};
        const int u = tid + p * nt;
        if (a.w && u < units) load_eight<VEC>(e, static_cast<const T*>(a.w), u, a.H);
        e.to_f32(w[p]);
        if (!a.w)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[p][i] = 1.0f;
    }
    int buf = 0;
    Eight<T> dy[PER] = {}, h[PER] = {}, dh[PER] = {};
    float rstd = 0.0f;
    // The next row's loads are in flight during this one's sum: a block has few rows at a time.
    auto load = [&](int64_t row, Eight<T>(&dy)[PER], Eight<T>(&h)[PER], Eight<T>(&dh)[PER], float& rstd) {
        if (row >= a.T) return;
        rstd = a.rstd[row];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int u = tid + p * nt;
            if (u < units) {
                load_eight<VEC>(dy[p], static_cast<const T*>(a.dy) + row * a.dy_stride, u, a.H);
                load_eight<VEC>(h[p], static_cast<const T*>(a.h) + row * a.h_stride, u, a.H);
                if (a.dh) load_eight<VEC>(dh[p], static_cast<const T*>(a.dh) + row * a.dh_stride, u, a.H);
            }
        }
    };
    load(part, dy, h, dh, rstd);
    for (int64_t row = part; row < a.T; row += a.parts) {
        Eight<T> dy2[PER] = {}, h2[PER] = {}, dh2[PER] = {};
        float rstd2 = 0.0f;
        load(row + a.parts, dy2, h2, dh2, rstd2);
        float dot = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            float d[8], x[8];
            dy[p].to_f32(d);
            h[p].to_f32(x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float g = d[i] * (x[i] * rstd);
                acc[p][i] += g;
                dot = fmaf(g, w[p][i], dot);
            }
        }
        const float mean = row_sum<ONE>(dot, s_part, buf) / (float)a.H;
        buf ^= 1;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int u = tid + p * nt;
            if (u >= units) break;
            float d[8], x[8], q[8];
            dy[p].to_f32(d);
            h[p].to_f32(x);
            dh[p].to_f32(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = fmaf(rstd, fmaf(-x[i] * rstd, mean, d[i] * w[p][i]), q[i]);
            Eight<T> o;
            o.from_f32(d);
            store_eight<VEC>(o, static_cast<T*>(a.dx) + row * a.dx_stride, u, a.H);
        }
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            dy[p] = dy2[p];
            h[p] = h2[p];
            dh[p] = dh2[p];
        }
        rstd = rstd2;
    }
    if (!a.dw || part >= a.parts) return;
    float* out = a.parts == 1 ? a.dw : a.ws + (int64_t)part * a.H;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int c = 8 * (tid + p * nt);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < a.H) out[c + i] = acc[p][i];
    }
}

// dw[c] = the sum of the parts' column c: 32 columns a block, each by eight threads of the block that
// take every eighth part.
__global__ void __launch_bounds__(256) norm_parts_kernel(const float* ws, int parts, int H, float* dw)
{
    __shared__ float s[8][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < H)
#pragma unroll 8
        for (int p = warp; p < parts; p += 8) v += ws[(int64_t)p * H + c];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < H) {
#pragma unroll
        for (int q = 1; q < 8; ++q) v += s[q][lane];
        dw[c] = v;
    }
}

template <typename T>
static NormKernel norm_of(int per, bool one, bool vec)
{
    if (one) return per == 1 ? (vec ? norm_kernel<T, 1, true, true> : norm_kernel<T, 1, true, false>)
                             : (vec ? norm_kernel<T, 2, true, true> : norm_kernel<T, 2, true, false>);
    return per == 1 ? (vec ? norm_kernel<T, 1, false, true> : norm_kernel<T, 1, false, false>)
                    : (vec ? norm_kernel<T, 2, false, true> : norm_kernel<T, 2, false, false>);
}

NormKernel norm_kernel_for(int dtype, int per, bool one, bool vec)
{
    switch (dtype) {
        case MOE_BF16: return norm_of<__nv_bfloat16>(per, one, vec);
        case MOE_FP16: return norm_of<__half>(per, one, vec);
        default: return norm_of<float>(per, one, vec);
    }
}

template <typename T, bool VEC>
static NormBackKernel norm_back_of(int per, bool one, int threads)
{
    if (one) return per == 1 ? norm_back_kernel<T, 1, true, VEC, 256> : norm_back_kernel<T, 2, true, VEC, 256>;
    return threads <= 512 ? norm_back_kernel<T, 2, false, VEC, 512> : norm_back_kernel<T, 2, false, VEC, 1024>;
}

NormBackKernel norm_back_kernel_for(int dtype, int per, bool one, bool vec, int threads)
{
    switch (dtype) {
        case MOE_BF16:
            return vec ? norm_back_of<__nv_bfloat16, true>(per, one, threads) : norm_back_of<__nv_bfloat16, false>(per, one, threads);
        case MOE_FP16: return vec ? norm_back_of<__half, true>(per, one, threads) : norm_back_of<__half, false>(per, one, threads);
        default: return vec ? norm_back_of<float, true>(per, one, threads) : norm_back_of<float, false>(per, one, threads);
    }
}

}  // namespace moe
