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
    const int64_t step = ONE ? (int64_t)gridDim.x * 8 : gridDim.x;
    int buf = 0;
    for (int64_t row = ONE ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x; row < a.T; row += step) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        Eight<T> e[PER] = {}, r[PER] = {};
#pragma unroll
        for (int p = 0; p < PER; ++p)
            if (tid + p * nt < units) {
                load_eight<VEC>(e[p], x, tid + p * nt, a.H);
                if (a.res)
                    load_eight<VEC>(r[p], static_cast<const T*>(a.res) + row * a.res_stride, tid + p * nt, a.H);
            }
        F2 v[PER][4], sums(0.0f);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            to_pairs(e[p], v[p]);
            if (a.res) {
                F2 q[4];
                to_pairs(r[p], q);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[p][i] = v[p][i] + q[i];
                // the stream holds h in its own type, and its norm is that of what it holds
                from_pairs(v[p], e[p]);
                to_pairs(e[p], v[p]);
                if (a.h && tid + p * nt < units)
                    store_eight<VEC>(e[p], static_cast<T*>(a.h) + row * a.h_stride, tid + p * nt, a.H);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sums = fma2(v[p][i], v[p][i], sums);
        }
        const float2 both = sums.get();
        const float sum = row_sum<ONE>(both.x + both.y, s_part, buf);
        buf ^= 1;
        const float rstd = rsqrtf(sum / (float)a.H + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int u = tid + p * nt;
            const bool in = u < units;
            if (u - lane >= units) break;  // (a warp's lanes stay together)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[p][i] = v[p][i] * F2(rstd);
            if (a.w) {
                Eight<T> w = {};
                if (in) load_eight<VEC>(w, static_cast<const T*>(a.w), u, a.H);
                F2 q[4];
                to_pairs(w, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[p][i] = v[p][i] * q[i];
            }
            if (a.y && in) {
                Eight<T> o;
                from_pairs(v[p], o);
                store_eight<VEC>(o, static_cast<T*>(a.y) + row * a.y_stride, u, a.H);
            }
            if (a.codes) {  // H % 32 == 0: a block's four lanes are in or out together
                float f[8], top = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 q = v[p][i].get();
                    f[2 * i] = q.x;
                    f[2 * i + 1] = q.y;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(f[i])));
                uint32_t m = __float_as_uint(top);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t s = mx_scale_byte<E4M3>(m, a.rule);
                // the scales of four blocks (16 lanes) in one word, zero past the row's end
                uint32_t word = in ? s << (8 * ((lane >> 2) & 3)) : 0u;
                word |= __shfl_xor_sync(0xffffffffu, word, 4);
                word |= __shfl_xor_sync(0xffffffffu, word, 8);
                if (!in) continue;
                const F2 scale(mx_encode_scale(s));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 q = (v[p][i] * scale).get();
                    f[2 * i] = q.x;
                    f[2 * i + 1] = q.y;
                }
                reinterpret_cast<uint2*>(a.codes)[row * units + u] = s == 255u ? E4M3::zero() : E4M3::encode(f);
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

// The same for rows in 16-byte pieces that a block takes: a.depth rows' loads are in flight, copied into
// shared memory where each thread reads what it copied itself (so no barrier is needed for them, and no
// registers hold them): a block has one row in its registers and its sum waits for all of them.
template <typename T, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 2 : 1) norm_back_ring_kernel(NormBackArgs a)
{
    constexpr int PER = 2, kPieces = (int)sizeof(T) / 2;  // eights of a thread, 16-byte pieces of an eight
    extern __shared__ uint4 s_ring[];                     // [depth][3][PER][kPieces][threads]
    __shared__ float s_part[2][32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, nt = blockDim.x, units = a.H >> 3, part = blockIdx.x;
    const int tensor = PER * kPieces * nt, stage = 3 * tensor;   // pieces
    auto copy = [&](int slot, int64_t row) {
        if (row < a.T) {
            const T* from[3] = {static_cast<const T*>(a.dy) + row * a.dy_stride,
                                static_cast<const T*>(a.h) + row * a.h_stride,
                                a.dh ? static_cast<const T*>(a.dh) + row * a.dh_stride : nullptr};
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (!from[x]) continue;
#pragma unroll
                for (int p = 0; p < PER; ++p)
                    if (tid + p * nt < units)
#pragma unroll
                        for (int q = 0; q < kPieces; ++q)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(
                                             s_ring + slot * stage + x * tensor + (p * kPieces + q) * nt + tid)),
                                         "l"(reinterpret_cast<const uint4*>(from[x] + 8 * (tid + p * nt)) + q)
                                         : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");   // (of no copies past the last row)
    };
    auto read = [&](int slot, int x, int p) {
        Eight<T> e;
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const uint4 v = s_ring[slot * stage + x * tensor + (p * kPieces + q) * nt + tid];
            e.w[4 * q] = v.x;
            e.w[4 * q + 1] = v.y;
            e.w[4 * q + 2] = v.z;
            e.w[4 * q + 3] = v.w;
        }
        return e;
    };
    for (int d = 0; d < a.depth; ++d) copy(d, part + (int64_t)d * a.parts);
    F2 acc[PER][4], w[PER][4];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        Eight<T> e = {};
        if (a.w && tid + p * nt < units) e.template load<true>(static_cast<const T*>(a.w) + 8 * (tid + p * nt));
        to_pairs(e, w[p]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[p][i] = F2(0.0f);
            if (!a.w) w[p][i] = F2(1.0f);
        }
    }
    int buf = 0, slot = 0, at = 0;
    float rstds = 0.0f;   // of 32 of the block's rows, one a lane
    for (int64_t row = part; row < a.T; row += a.parts, at = (at + 1) & 31) {
        if (at == 0) {
            const int64_t mine = row + (int64_t)(tid & 31) * a.parts;
            rstds = mine < a.T ? a.rstd[mine] : 0.0f;
        }
        const float rstd = __shfl_sync(0xffffffffu, rstds, at);
        // (the thread's own copies of the oldest row have landed)
        if (a.depth == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (a.depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 2;" ::: "memory");
        F2 d[PER][4], x[PER][4], dot(0.0f);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            if (tid + p * nt >= units) {
#pragma unroll
                for (int i = 0; i < 4; ++i) d[p][i] = x[p][i] = F2(0.0f);
                continue;
            }
            to_pairs(read(slot, 0, p), d[p]);
            to_pairs(read(slot, 1, p), x[p]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[p][i] = x[p][i] * F2(rstd);
                acc[p][i] = fma2(d[p][i], x[p][i], acc[p][i]);
                d[p][i] = d[p][i] * w[p][i];
                dot = fma2(d[p][i], x[p][i], dot);
            }
        }
        const float2 both = dot.get();
        const float mean = row_sum<false>(both.x + both.y, s_part, buf) / (float)a.H;
        buf ^= 1;
        const F2 less(-mean), r(rstd);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            if (tid + p * nt >= units) break;
            F2 q[4];
            if (a.dh) to_pairs(read(slot, 2, p), q);
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!a.dh) q[i] = F2(0.0f);
                const float2 v = fma2(r, fma2(x[p][i], less, d[p][i]), q[i]).get();
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
            Eight<T> o;
            o.from_f32(f);
            o.store(static_cast<T*>(a.dx) + row * a.dx_stride + 8 * (tid + p * nt));
        }
        copy(slot, row + (int64_t)a.depth * a.parts);   // (over what this thread has read)
        slot = slot + 1 == a.depth ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!a.dw) return;
    float* out = a.parts == 1 ? a.dw : a.ws + (int64_t)part * a.H;
#pragma unroll
    for (int p = 0; p < PER; ++p)
        if (tid + p * nt < units)
#pragma unroll
            for (int i = 0; i < 4; ++i)   // (dw itself need not be aligned to more than an element)
                if (a.parts == 1) {
                    const float2 v = acc[p][i].get();
                    out[8 * (tid + p * nt) + 2 * i] = v.x;
                    out[8 * (tid + p * nt) + 2 * i + 1] = v.y;
                } else {
                    reinterpret_cast<uint64_t*>(out)[4 * (tid + p * nt) + i] = acc[p][i].v;
                }
}

// dw[c] = the sum of the parts' column c: 32 columns a block, each by 32 threads that take every 32nd part.
__global__ void __launch_bounds__(1024) norm_parts_kernel(const float* ws, int parts, int H, float* dw)
{
    __shared__ float s[32][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < H)
#pragma unroll 8
        for (int p = warp; p < parts; p += 32) v += ws[(int64_t)p * H + c];
    s[warp][lane] = v;
    __syncthreads();
    v = s[lane][warp];   // column `warp` of the block's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * 32 + warp < H) dw[blockIdx.x * 32 + warp] = v;
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

template <typename T>
static NormBackKernel norm_back_of(int per, bool one, bool vec, int threads)
{
    if (one && per == 1) return vec ? norm_back_kernel<T, 1, true, true, 256> : norm_back_kernel<T, 1, true, false, 256>;
    if (one) return vec ? norm_back_kernel<T, 2, true, true, 256> : norm_back_kernel<T, 2, true, false, 256>;
    if (vec)
        return threads <= 256 ? norm_back_ring_kernel<T, 256>
             : threads <= 512 ? norm_back_ring_kernel<T, 512> : norm_back_ring_kernel<T, 1024>;
    return threads <= 512 ? norm_back_kernel<T, 2, false, false, 512> : norm_back_kernel<T, 2, false, false, 1024>;
}

NormBackKernel norm_back_kernel_for(int dtype, int per, bool one, bool vec, int threads)
{
    switch (dtype) {
        case MOE_BF16: return norm_back_of<__nv_bfloat16>(per, one, vec, threads);
        case MOE_FP16: return norm_back_of<__half>(per, one, vec, threads);
        default: return norm_back_of<float>(per, one, vec, threads);
    }
}

}  // namespace moe
