// Root-mean-square norm with the residual's addition, its result in the rows' own type and as an MXFP8
// matrix, and its gradient.
//
// Rows of over 512 elements in 16-byte pieces have a block each at a time (16 elements a thread), and each
// SM as many blocks as its registers hold: the rows to come are copied into a ring in shared memory, where a
// thread reads what it copied itself, so that no barrier is needed for them and no registers hold them while
// the row's sum waits for all of its threads.  Short rows (the gradient's up to 1024 16-bit elements) have a
// warp each; rows that are in no 16-byte pieces are read an element, or two 16-bit ones, a lane at a time.
//
// Rows of 4096 and 8192 elements are bound by memory, from 0.8 of the measured copy rate up: 8192 x 4096 bf16 with
// residual, h, y and MXFP8 50 us (6.0 TB/s; fp32 86), y alone 25 us, its gradient 46 us (5.8 TB/s; fp32 83, 6.5
// TB/s).  Others come to 0.5 to 0.7 of it: 16384 x 512 15 us each way; the gradient of 8192 x 1024 20 us and of
// x 2048 32 us, with few rows a warp or block before the parts of the weight's gradient are added up; that of
// 2048 x 16384 68 us, where a block of 1024 threads is alone on its SM and nothing hides its barrier.  What is in
// no 16 bytes is bound by its instructions: 8192 x 4097 bf16 72 us with residual, h and y, its gradient 101.
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

// ---- rows of which a thread holds eights in registers

// The elements of eight u (of a warp's 256 u / 32 ..): in a row, as 16 bytes (kVec) or one by one (kEach); or
// those 32 (kApart), in pairs of 16-bit ones 64 (kPairs) apart, so that a warp's accesses are contiguous
// (8192 x 4097 bf16 with the residual, h and y: 184 us one by one).
enum Mode { kVec, kEach, kApart, kPairs };

template <int MODE>
__device__ __forceinline__ int element(int u, int i)
{
    if constexpr (MODE == kApart) return (u >> 5) * 256 + (u & 31) + 32 * i;
    else if constexpr (MODE == kPairs) return (u >> 5) * 256 + 2 * (u & 31) + 64 * (i >> 1) + (i & 1);
    else return 8 * u + i;
}

template <int MODE, typename T>
__device__ __forceinline__ void load_eight(Eight<T>& e, const T* row, int u, int H)
{
    if constexpr (MODE == kVec) {
        e.template load<true>(row + 8 * u);
    } else if constexpr (MODE == kEach) {
        e.load_some(row + 8 * u, H - 8 * u);
    } else {
#pragma unroll
        for (int q = 0; q < Eight<T>::kWords; ++q) {
            e.w[q] = 0;
            if constexpr (MODE == kPairs || sizeof(T) == 4) {
                const int c = element<MODE>(u, sizeof(T) == 4 ? q : 2 * q);
                if (c < H) e.w[q] = *reinterpret_cast<const uint32_t*>(row + c);
            } else {
                const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
                const int c = element<MODE>(u, 2 * q), d = element<MODE>(u, 2 * q + 1);
                if (c < H) e.w[q] = h[c];
                if (d < H) e.w[q] |= (uint32_t)h[d] << 16;
            }
        }
    }
}

template <int MODE, typename T>
__device__ __forceinline__ void store_eight(const Eight<T>& e, T* row, int u, int H)
{
    if constexpr (MODE == kVec) {
        e.store(row + 8 * u);
    } else if constexpr (MODE == kEach) {
        e.store_some(row + 8 * u, H - 8 * u);
    } else {
#pragma unroll
        for (int q = 0; q < Eight<T>::kWords; ++q) {
            if constexpr (MODE == kPairs || sizeof(T) == 4) {
                const int c = element<MODE>(u, sizeof(T) == 4 ? q : 2 * q);
                if (c < H) *reinterpret_cast<uint32_t*>(row + c) = e.w[q];
            } else {
                uint16_t* h = reinterpret_cast<uint16_t*>(row);
                const int c = element<MODE>(u, 2 * q), d = element<MODE>(u, 2 * q + 1);
                if (c < H) h[c] = (uint16_t)e.w[q];
                if (d < H) h[d] = (uint16_t)(e.w[q] >> 16);
            }
        }
    }
}

// ---- rows of which a thread holds 16-byte pieces, every blockDim.x-th one

template <typename T>
struct Piece {
    static constexpr int kOf = 16 / (int)sizeof(T);  // elements
    static constexpr int kPer = (int)sizeof(T);      // pieces of a thread: 16 elements
    F2 v[kOf / 2];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kOf / 2; ++i) v[i] = F2(0.0f);
    }
    __device__ __forceinline__ void from(uint4 r)
    {
        if constexpr (sizeof(T) == 4) {
            v[0] = F2(__uint_as_float(r.x), __uint_as_float(r.y));
            v[1] = F2(__uint_as_float(r.z), __uint_as_float(r.w));
        } else {
            Eight<T> e;
            e.w[0] = r.x;
            e.w[1] = r.y;
            e.w[2] = r.z;
            e.w[3] = r.w;
            to_pairs(e, v);
        }
    }
    __device__ __forceinline__ uint4 to() const
    {
        if constexpr (sizeof(T) == 4) {
            const float2 a = v[0].get(), b = v[1].get();
            return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
        } else {
            Eight<T> e;
            from_pairs(v, e);
            return make_uint4(e.w[0], e.w[1], e.w[2], e.w[3]);
        }
    }
};

// The block's ring: `depth` rows (ONE: of each of its warps) of TENSORS tensors, [depth][TENSORS][PER][threads]
// pieces.
template <typename T, int TENSORS, int PER, bool ONE>
struct Ring {
    uint4* at;
    int depth, pieces;   // rows; pieces of a row
    // piece k of this thread
    static __device__ __forceinline__ int piece(int k)
    {
        return ONE ? (int)(threadIdx.x & 31) + 32 * k : (int)threadIdx.x + k * (int)blockDim.x;
    }
    __device__ __forceinline__ uint4* place(int slot, int x, int k) const
    {
        return at + ((slot * TENSORS + x) * PER + k) * blockDim.x + threadIdx.x;
    }
    // Copies this thread's pieces of a row (null: of no row), and counts them as one group.
    __device__ __forceinline__ void copy(int slot, const T* const (&from)[TENSORS]) const
    {
#pragma unroll
        for (int x = 0; x < TENSORS; ++x) {
            if (!from[x]) continue;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int c = piece(k);
                if (c < pieces)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(place(slot, x, k))),
                                 "l"(reinterpret_cast<const uint4*>(from[x]) + c)
                                 : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // The oldest group has landed.
    __device__ __forceinline__ void wait() const
    {
        if (depth == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 2;" ::: "memory");
    }
};

}  // namespace

// A row in the registers of one warp (ONE, eight rows a block) or of one block, PER eights a thread: each
// input is read once and each output written once.
template <typename T, int PER, bool ONE, int MODE>
__global__ void __launch_bounds__(ONE ? 256 : 1024) norm_kernel(NormArgs a)
{
    __shared__ float s_part[2][32];
    pdl_wait();
    pdl_trigger();
    const int tid = ONE ? threadIdx.x & 31 : threadIdx.x, nt = ONE ? 32 : blockDim.x;
    const int lane = threadIdx.x & 31;
    const int blocks = a.H >> 5, KA = (blocks + 3) >> 2;
    const int64_t step = ONE ? (int64_t)gridDim.x * 8 : gridDim.x;
    int buf = 0;
    for (int64_t row = ONE ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x; row < a.T; row += step) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        Eight<T> e[PER] = {}, r[PER] = {};
#pragma unroll
        for (int p = 0; p < PER; ++p)
            if (element<MODE>(tid + p * nt, 0) < a.H) {
                load_eight<MODE>(e[p], x, tid + p * nt, a.H);
                if (a.res)
                    load_eight<MODE>(r[p], static_cast<const T*>(a.res) + row * a.res_stride, tid + p * nt, a.H);
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
                if (a.h && element<MODE>(tid + p * nt, 0) < a.H)
                    store_eight<MODE>(e[p], static_cast<T*>(a.h) + row * a.h_stride, tid + p * nt, a.H);
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
            const bool in = element<MODE>(u, 0) < a.H;
            if (8 * (u - lane) >= a.H) break;  // (a warp's lanes stay together)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[p][i] = v[p][i] * F2(rstd);
            if (a.w) {
                Eight<T> w = {};
                if (in) load_eight<MODE>(w, static_cast<const T*>(a.w), u, a.H);
                F2 q[4];
                to_pairs(w, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[p][i] = v[p][i] * q[i];
            }
            if (a.y && in) {
                Eight<T> o;
                from_pairs(v[p], o);
                store_eight<MODE>(o, static_cast<T*>(a.y) + row * a.y_stride, u, a.H);
            }
            if constexpr (MODE == kVec || MODE == kEach) {
                if (!a.codes) continue;  // (H % 32 == 0: a block's four lanes are in or out together)
                float f[8], top = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) top = max_nan(top, v[p][i]);
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
                reinterpret_cast<uint2*>(a.codes)[row * (a.H >> 3) + u] = s == 255u ? E4M3::zero() : E4M3::encode(f);
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

// A block a row, the rows to come in the ring.
template <typename T, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 3 : 1) norm_ring_kernel(NormArgs a)
{
    using P = Piece<T>;
    constexpr int kPer = P::kPer, kOf = P::kOf, kLanes = 32 / kOf;  // lanes of a block of 32
    extern __shared__ uint4 s_ring[];
    __shared__ float s_part[2][32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
    const Ring<T, 2, kPer, false> ring{s_ring, a.depth, a.H / kOf};
    const int blocks = a.H >> 5, KA = (blocks + 3) >> 2;
    auto copy = [&](int slot, int64_t row) {
        const bool in = row < a.T;
        ring.copy(slot, {in ? static_cast<const T*>(a.x) + row * a.x_stride : nullptr,
                         in && a.res ? static_cast<const T*>(a.res) + row * a.res_stride : nullptr});
    };
    for (int d = 0; d < a.depth; ++d) copy(d, blockIdx.x + (int64_t)d * gridDim.x);
    uint4 w[kPer] = {};   // (as they are: as pairs they take twice the registers, and the SM a block less)
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (a.w && tid + k * nt < ring.pieces) w[k] = static_cast<const uint4*>(a.w)[tid + k * nt];
    int buf = 0, slot = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        ring.wait();
        P v[kPer];
        F2 sums(0.0f);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            v[k].zero();
            if (tid + k * nt >= ring.pieces) continue;
            v[k].from(*ring.place(slot, 0, k));
            if (a.res) {
                P r;
                r.from(*ring.place(slot, 1, k));
#pragma unroll
                for (int i = 0; i < kOf / 2; ++i) v[k].v[i] = v[k].v[i] + r.v[i];
                // the stream holds h in its own type, and its norm is that of what it holds
                const uint4 h = v[k].to();
                v[k].from(h);
                if (a.h)
                    reinterpret_cast<uint4*>(static_cast<T*>(a.h) + row * a.h_stride)[tid + k * nt] = h;
            }
#pragma unroll
            for (int i = 0; i < kOf / 2; ++i) sums = fma2(v[k].v[i], v[k].v[i], sums);
        }
        copy(slot, row + (int64_t)a.depth * gridDim.x);   // (over what this thread has read)
        slot = slot + 1 == a.depth ? 0 : slot + 1;
        const float2 both = sums.get();
        const float sum = row_sum<false>(both.x + both.y, s_part, buf);
        buf ^= 1;
        const float rstd = rsqrtf(sum / (float)a.H + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int c = tid + k * nt;
            const bool in = c < ring.pieces;
            if (c - lane >= ring.pieces) break;  // (a warp's lanes stay together)
#pragma unroll
            for (int i = 0; i < kOf / 2; ++i) v[k].v[i] = v[k].v[i] * F2(rstd);
            if (a.w) {
                P q;
                q.from(w[k]);
#pragma unroll
                for (int i = 0; i < kOf / 2; ++i) v[k].v[i] = v[k].v[i] * q.v[i];
            }
            if (a.y && in) reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * a.y_stride)[c] = v[k].to();
            if (!a.codes) continue;  // (H % 32 == 0: a block's lanes are in or out together)
            float f[kOf], top = 0.0f;
#pragma unroll
            for (int i = 0; i < kOf / 2; ++i) top = max_nan(top, v[k].v[i]);
            uint32_t m = __float_as_uint(top);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const uint32_t s = mx_scale_byte<E4M3>(m, a.rule);
            // the scales of four blocks in one word, zero past the row's end
            uint32_t word = in ? s << (8 * ((lane / kLanes) & 3)) : 0u;
            word |= __shfl_xor_sync(0xffffffffu, word, kLanes);
            word |= __shfl_xor_sync(0xffffffffu, word, 2 * kLanes);
            if (!in) continue;
            const F2 scale(mx_encode_scale(s));
#pragma unroll
            for (int i = 0; i < kOf / 2; ++i) {
                const float2 q = (v[k].v[i] * scale).get();
                f[2 * i] = q.x;
                f[2 * i + 1] = q.y;
            }
            const int64_t at = row * ring.pieces + c;
            if constexpr (kOf == 8) reinterpret_cast<uint2*>(a.codes)[at] = s == 255u ? E4M3::zero() : E4M3::encode(f);
            else reinterpret_cast<uint32_t*>(a.codes)[at] = s == 255u ? 0u : f32x4_to_e4m3(f);
            const int kb = c / kLanes;
            if (a.layout == MOE_SF_TILED) {
                if (lane % (4 * kLanes) == 0)
                    *reinterpret_cast<uint32_t*>(a.sf + mx_sf_tiled(0, 0, KA, (int)row, kb)) = word;
            } else if (lane % kLanes == 0) {
                a.sf[row * blocks + kb] = (uint8_t)s;
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// With d = dy w and x^ = h rstd: dx = rstd (d - x^ mean(d x^)) + dh, dw = sum over the rows of dy x^.  A
// block (ONE: each of its eight warps) takes every (number of parts)-th row and holds its part of dw in
// registers; the parts are added up in order by norm_parts_kernel, so results do not change from call to call.
template <typename T, int PER, bool ONE, int MODE, int NT>
__global__ void __launch_bounds__(NT, NT == 320 ? 2 : 1) norm_back_kernel(NormBackArgs a)
{
    __shared__ float s_part[2][32];
    __shared__ float s_dw[ONE ? 8 * 256 * PER : 1];
    pdl_wait();
    pdl_trigger();
    const int tid = ONE ? threadIdx.x & 31 : threadIdx.x, nt = ONE ? 32 : blockDim.x;
    const int64_t first = ONE ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x, step = ONE ? a.parts * 8 : a.parts;
    float acc[PER][8] = {}, w[PER][8];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        Eight<T> e = {};
        const int u = tid + p * nt;
        if (a.w && element<MODE>(u, 0) < a.H) load_eight<MODE>(e, static_cast<const T*>(a.w), u, a.H);
        e.to_f32(w[p]);
        if (!a.w)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[p][i] = 1.0f;
    }
    int buf = 0;
    for (int64_t row = first; row < a.T; row += step) {
        Eight<T> dy[PER] = {}, h[PER] = {}, dh[PER] = {};
        const float rstd = a.rstd[row];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int u = tid + p * nt;
            if (element<MODE>(u, 0) < a.H) {
                load_eight<MODE>(dy[p], static_cast<const T*>(a.dy) + row * a.dy_stride, u, a.H);
                load_eight<MODE>(h[p], static_cast<const T*>(a.h) + row * a.h_stride, u, a.H);
                if (a.dh) load_eight<MODE>(dh[p], static_cast<const T*>(a.dh) + row * a.dh_stride, u, a.H);
            }
        }
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
            if (element<MODE>(u, 0) >= a.H) break;
            float d[8], x[8], q[8];
            dy[p].to_f32(d);
            h[p].to_f32(x);
            dh[p].to_f32(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = fmaf(rstd, fmaf(-x[i] * rstd, mean, d[i] * w[p][i]), q[i]);
            Eight<T> o;
            o.from_f32(d);
            store_eight<MODE>(o, static_cast<T*>(a.dx) + row * a.dx_stride, u, a.H);
        }
    }
    if (!a.dw) return;
    float* out = a.parts == 1 ? a.dw : a.ws + (int64_t)blockIdx.x * a.H;
    float* to = ONE ? s_dw + (threadIdx.x >> 5) * 256 * PER : out;
#pragma unroll
    for (int p = 0; p < PER; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = element<MODE>(tid + p * nt, i);
            if (c < a.H) to[c] = acc[p][i];
        }
    if constexpr (ONE) {
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += 256) {
            float v = s_dw[c];
#pragma unroll
            for (int q = 1; q < 8; ++q) v += s_dw[q * 256 * PER + c];
            out[c] = v;
        }
    }
}

// The same with the rows to come in the ring, PER pieces a thread.
template <typename T, int PER, bool ONE, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 2 : 1) norm_back_ring_kernel(NormBackArgs a)
{
    using P = Piece<T>;
    constexpr int kOf = P::kOf;
    extern __shared__ uint4 s_ring[];
    __shared__ float s_part[2][32];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5;
    const int64_t first = ONE ? blockIdx.x * 8 + warp : blockIdx.x, step = ONE ? a.parts * 8 : a.parts;
    const Ring<T, 3, PER, ONE> ring{s_ring, a.depth, a.H / kOf};
    auto copy = [&](int slot, int64_t row) {
        const bool in = row < a.T;
        ring.copy(slot, {in ? static_cast<const T*>(a.dy) + row * a.dy_stride : nullptr,
                         in ? static_cast<const T*>(a.h) + row * a.h_stride : nullptr,
                         in && a.dh ? static_cast<const T*>(a.dh) + row * a.dh_stride : nullptr});
    };
    for (int d = 0; d < a.depth; ++d) copy(d, first + d * step);
    P acc[PER];
    uint4 w[PER] = {};
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        acc[k].zero();
        if (a.w && ring.piece(k) < ring.pieces) w[k] = static_cast<const uint4*>(a.w)[ring.piece(k)];
    }
    int buf = 0, slot = 0, at = 0;
    float rstds = 0.0f;   // of 32 of the rows to come, one a lane (a load a row would be waited for each time)
    for (int64_t row = first; row < a.T; row += step, at = (at + 1) & 31) {
        if (at == 0) {
            const int64_t mine = row + (int64_t)(threadIdx.x & 31) * step;
            rstds = mine < a.T ? a.rstd[mine] : 0.0f;
        }
        const float rstd = __shfl_sync(0xffffffffu, rstds, at);
        ring.wait();
        P d[PER], x[PER];
        F2 dot(0.0f);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            d[k].zero();
            x[k].zero();
            if (ring.piece(k) >= ring.pieces) continue;
            d[k].from(*ring.place(slot, 0, k));
            x[k].from(*ring.place(slot, 1, k));
            P q;
            q.from(w[k]);
#pragma unroll
            for (int i = 0; i < kOf / 2; ++i) {
                x[k].v[i] = x[k].v[i] * F2(rstd);
                acc[k].v[i] = fma2(d[k].v[i], x[k].v[i], acc[k].v[i]);
                if (a.w) d[k].v[i] = d[k].v[i] * q.v[i];
                dot = fma2(d[k].v[i], x[k].v[i], dot);
            }
        }
        const float2 both = dot.get();
        const float mean = row_sum<ONE>(both.x + both.y, s_part, buf) / (float)a.H;
        buf ^= 1;
        const F2 less(-mean), r(rstd);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (ring.piece(k) >= ring.pieces) break;
            P q;
            q.zero();
            if (a.dh) q.from(*ring.place(slot, 2, k));
#pragma unroll
            for (int i = 0; i < kOf / 2; ++i) q.v[i] = fma2(r, fma2(x[k].v[i], less, d[k].v[i]), q.v[i]);
            reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + row * a.dx_stride)[ring.piece(k)] = q.to();
        }
        copy(slot, row + a.depth * step);   // (over what this thread has read)
        slot = slot + 1 == a.depth ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!a.dw) return;
    float* out = a.parts == 1 ? a.dw : a.ws + (int64_t)blockIdx.x * a.H;
    float* s_dw = reinterpret_cast<float*>(s_ring);   // ONE: [8][H], in the ring's place
    if constexpr (ONE) __syncthreads();
    float* to = ONE ? s_dw + warp * a.H : out;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int c = ring.piece(k);
        if (c >= ring.pieces) break;
#pragma unroll
        for (int i = 0; i < kOf / 2; ++i)   // (dw itself need not be aligned to more than an element)
            if (!ONE && a.parts == 1) {
                const float2 v = acc[k].v[i].get();
                to[kOf * c + 2 * i] = v.x;
                to[kOf * c + 2 * i + 1] = v.y;
            } else {
                reinterpret_cast<uint64_t*>(to)[kOf / 2 * c + i] = acc[k].v[i].v;
            }
    }
    if constexpr (ONE) {
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += 256) {
            float v = s_dw[c];
#pragma unroll
            for (int q = 1; q < 8; ++q) v += s_dw[q * a.H + c];
            out[c] = v;
        }
    }
}

// dw[c] = the sum of the parts' column c: eight columns (a 32-byte sector) a block, each by 32 threads that
// take every 32nd part.
__global__ void __launch_bounds__(256) norm_parts_kernel(const float* ws, int parts, int H, float* dw)
{
    __shared__ float s[8][33];
    pdl_wait();
    pdl_trigger();
    const int column = threadIdx.x & 7, l = threadIdx.x >> 3, c = blockIdx.x * 8 + column;
    float v = 0.0f;
    if (c < H)
#pragma unroll 8
        for (int p = l; p < parts; p += 32) v += ws[(int64_t)p * H + c];
    s[column][l] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;   // column `warp` of the block's
    v = s[warp][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * 8 + warp < H) dw[blockIdx.x * 8 + warp] = v;
}

// (MXFP8 results of rows that are in no 16 bytes: one by one.  Long rows in 16-byte pieces get here in fp32 with
// a residual alone, all others go through the ring.)
template <typename T, int PER, bool ONE>
static NormKernel norm_of(int piece, bool codes)
{
    if constexpr (ONE || sizeof(T) == 4)
        if (piece == 16) return norm_kernel<T, PER, ONE, kVec>;
    if (codes) return norm_kernel<T, PER, ONE, kEach>;
    if (sizeof(T) == 2 && piece >= 4) return norm_kernel<T, PER, ONE, sizeof(T) == 2 ? kPairs : kApart>;
    return norm_kernel<T, PER, ONE, kApart>;
}

template <typename T>
static NormKernel norm_of(int H, int piece, bool codes, int threads, bool ring)
{
    if (H <= 256) return norm_of<T, 1, true>(piece, codes);
    if (H <= 512) return norm_of<T, 2, true>(piece, codes);
    if (ring) return threads <= 256 ? norm_ring_kernel<T, 256> : norm_ring_kernel<T, 1024>;
    return norm_of<T, 2, false>(piece, codes);
}

NormKernel norm_kernel_for(int dtype, int H, int piece, bool codes, int threads, bool ring)
{
    switch (dtype) {
        case MOE_BF16: return norm_of<__nv_bfloat16>(H, piece, codes, threads, ring);
        case MOE_FP16: return norm_of<__half>(H, piece, codes, threads, ring);
        default: return norm_of<float>(H, piece, codes, threads, ring);
    }
}

template <typename T, int PER, bool ONE, int NT>
static NormBackKernel norm_back_of(int piece)
{
    if (sizeof(T) == 2 && piece >= 4) return norm_back_kernel<T, PER, ONE, sizeof(T) == 2 ? kPairs : kApart, NT>;
    return norm_back_kernel<T, PER, ONE, kApart, NT>;
}

template <typename T>
static NormBackKernel norm_back_of(int H, int piece, int threads)
{
    constexpr int kPer = Piece<T>::kPer;
    if (piece == 16) {
        if (H <= kNormShort) return norm_back_ring_kernel<T, kPer, true, 256>;
        if (sizeof(T) == 2 && H <= 2 * kNormShort) return norm_back_ring_kernel<T, 4, true, 256>;
        return threads <= 256 ? norm_back_ring_kernel<T, kPer, false, 256>
             : threads <= 512 ? norm_back_ring_kernel<T, kPer, false, 512> : norm_back_ring_kernel<T, kPer, false, 1024>;
    }
    if (H <= 256) return norm_back_of<T, 1, true, 256>(piece);
    if (H <= kNormShort) return norm_back_of<T, 2, true, 256>(piece);
    return threads <= 320 ? norm_back_of<T, 2, false, 320>(piece) : norm_back_of<T, 2, false, 1024>(piece);
}

NormBackKernel norm_back_kernel_for(int dtype, int H, int piece, int threads)
{
    switch (dtype) {
        case MOE_BF16: return norm_back_of<__nv_bfloat16>(H, piece, threads);
        case MOE_FP16: return norm_back_of<__half>(H, piece, threads);
        default: return norm_back_of<float>(H, piece, threads);
    }
}

}  // namespace moe
