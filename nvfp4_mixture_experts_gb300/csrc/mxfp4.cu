// MXFP4 and MXFP8: quantisation (MXFP4 also of a matrix's transpose) and the tiled scale layout.
#include "mx.cuh"

namespace moe {

namespace {

// Stores the scale bytes of blocks kb .. kb + 3 of row r (kb a multiple of 4; the bytes of blocks
// past the row's end are zero, as the tiled layout wants them).
__device__ __forceinline__ void store_scales(uint8_t* sf, int layout, int64_t b, int R, int r,
                                             int blocks, int kb, uint32_t word)
{
    if (layout == MOE_SF_TILED) {
        *reinterpret_cast<uint32_t*>(sf + mx_sf_tiled(b, div_up(R, 128), (blocks + 3) >> 2, r, kb)) = word;
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
// together.  8192 x 4096 bf16: 24.3 us with values (152 MB, 6.2 TB/s: memory), 15.5 without (85 MB, 5.5
// TB/s: the issue slots; MXFP8 16.3, 6.2 TB/s); fp32 with values 43.6 us (6.6 TB/s).  A run loaded ahead of the work on the
// one before took 99 registers and 17.8 us without values, the same with.
template <typename F, typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_quant_kernel(MxQuantArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kPer = kMxQuantRun / 32;
    const int lane = threadIdx.x & 31;
    const int units = a.cols >> 3;  // eights per row, a multiple of 4
    const int runs = (units + kMxQuantRun - 1) / kMxQuantRun;
    const uint32_t items = (uint32_t)a.batch * a.rows * runs;  // (fits: checked by the caller)
    const uint32_t step = gridDim.x * (blockDim.x >> 5);
    const int blocks = units >> 2, RB = div_up(a.rows, 128), KA = (blocks + 3) >> 2;
    for (uint64_t i0 = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i0 < items; i0 += step) {
        const uint32_t i = (uint32_t)i0;
        const uint32_t row = i / (uint32_t)runs;                    // of all matrices
        const int u0 = (int)(i - row * runs) * kMxQuantRun + lane;  // this lane's first eight
        const int b = a.batch == 1 ? 0 : (int)(row / (uint32_t)a.rows);
        const int r = (int)(row - (uint32_t)b * a.rows);
        if (a.perm_src && a.perm_src[r] < 0) continue;
        const T* x = static_cast<const T*>(a.x) + b * a.batch_stride + r * a.row_stride + u0 * 8;
        Eight<T> e[kPer] = {};
#pragma unroll
        for (int p = 0; p < kPer; ++p)
            if (u0 + 32 * p < units) e[p].template load<VEC>(x + 256 * p);
        const int64_t at = (int64_t)row * units + u0;
        typename F::Codes* codes_at = reinterpret_cast<typename F::Codes*>(a.codes) + at;
        T* values_at = static_cast<T*>(a.values) + at * 8;
        // the scale word of this lane's first block's atom (tiled), or its scale byte
        const int kb = u0 >> 2;
        uint8_t* sf_at = a.sf + (a.layout == MOE_SF_TILED ? mx_sf_tiled(b, RB, KA, r, kb)
                                                          : (size_t)row * blocks + kb);
        // piece p of the run; the bytes of blocks past the row's end are zero in the tiled layout
        auto piece = [&](int p, bool in) {
            const uint32_t s = mx_scale_byte<F>(e[p].amax4(), a.rule);
            // the scales of four blocks (16 lanes) in one word
            uint32_t word = in ? s << (8 * ((lane >> 2) & 3)) : 0u;
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            word |= __shfl_xor_sync(0xffffffffu, word, 8);
            if (!in) return;
            F2 w[4];
            float v[8];
            to_pairs(e[p], w);
            const F2 scale(mx_encode_scale(s));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 f = (w[q] * scale).get();
                v[2 * q] = f.x;
                v[2 * q + 1] = f.y;
            }
            const typename F::Codes codes = s == 255u ? F::zero() : F::encode(v);
            codes_at[32 * p] = codes;
            // 8 blocks, two atoms, per 32 eights
            if (a.layout == MOE_SF_TILED) {
                if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(sf_at + 1024 * p) = word;
            } else if ((lane & 3) == 0) {
                sf_at[8 * p] = (uint8_t)s;
            }
            if (a.values) {
                const float d = mx_decode_scale(s);
                F::decode(codes, v);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= d;
                Eight<T> o;
                o.from_f32(v);
                o.store(values_at + 256 * p);
            }
        };
        // (a block's four lanes are in or out together)
        if (u0 - lane + kMxQuantRun <= units) {
#pragma unroll
            for (int p = 0; p < kPer; ++p) piece(p, true);
        } else {
#pragma unroll
            for (int p = 0; p < kPer; ++p)
                if (u0 - lane + 32 * p < units) piece(p, u0 + 32 * p < units);
        }
    }
}

// The same for short rows and small matrices: a thread per eight elements of all rows, so that a warp
// is full whatever a row's length; a block's first thread stores its scale byte.  262144 x 32 bf16
// with values: 9.5 us (38 MB, half of it in L2); 1 x 4096: 1.5 us (the launch).
template <typename F, typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_quant_short_kernel(MxQuantArgs a)
{
    pdl_wait();
    pdl_trigger();
    const uint32_t units = a.cols >> 3, blocks = units >> 2;
    const uint32_t n = (uint32_t)a.batch * a.rows * units;  // (fits: checked by the caller)
    const int RB = div_up(a.rows, 128), KA = ((int)blocks + 3) >> 2;
    for (uint64_t i0 = blockIdx.x * 256u; i0 < n; i0 += gridDim.x * 256u) {
        const uint64_t i = i0 + threadIdx.x;
        const uint32_t at_most = (uint32_t)min(i, (uint64_t)n - 1);
        const uint32_t row = at_most / units;
        const int u = (int)(at_most - row * units);
        const int b = a.batch == 1 ? 0 : (int)(row / (uint32_t)a.rows), r = (int)(row - (uint32_t)b * a.rows);
        const bool live = i < n && !(a.perm_src && a.perm_src[r] < 0);
        Eight<T> e = {};
        if (live)
            e.template load<VEC>(static_cast<const T*>(a.x) + b * a.batch_stride + r * a.row_stride + u * 8);
        const uint32_t s = mx_scale_byte<F>(e.amax4(), a.rule);
        if (!live) continue;
        float v[8];
        e.to_f32(v);
        const float scale = mx_encode_scale(s);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= scale;
        const typename F::Codes codes = s == 255u ? F::zero() : F::encode(v);
        reinterpret_cast<typename F::Codes*>(a.codes)[i] = codes;
        if ((u & 3) == 0) {
            const int kb = u >> 2;
            if (a.layout == MOE_SF_CANONICAL) {
                a.sf[(size_t)row * blocks + kb] = (uint8_t)s;
            } else {  // the last block also zeroes the scales past it in its atom
                uint8_t* at = a.sf + mx_sf_tiled(b, RB, KA, r, kb);
                at[0] = (uint8_t)s;
                if (kb == (int)blocks - 1)
                    for (int z = 1; z < 4 - (kb & 3); ++z) at[z] = 0;
            }
        }
        if (a.values) {
            const float d = mx_decode_scale(s);
            F::decode(codes, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= d;
            e.from_f32(v);
            e.store(static_cast<T*>(a.values) + i * 8);
        }
    }
}

template <typename F, typename T>
static MxQuantKernel mx_quant_of(bool vec, bool short_rows)
{
    if (short_rows) return vec ? mx_quant_short_kernel<F, T, true> : mx_quant_short_kernel<F, T, false>;
    return vec ? mx_quant_kernel<F, T, true> : mx_quant_kernel<F, T, false>;
}

template <typename F>
static MxQuantKernel mx_quant_of(int dtype, bool vec, bool short_rows)
{
    switch (dtype) {
        case MOE_BF16: return mx_quant_of<F, __nv_bfloat16>(vec, short_rows);
        case MOE_FP16: return mx_quant_of<F, __half>(vec, short_rows);
        default: return mx_quant_of<F, float>(vec, short_rows);
    }
}

MxQuantKernel mx_quant_kernel_for(bool eight_bits, int dtype, bool vec, bool short_rows)
{
    return eight_bits ? mx_quant_of<E4M3>(dtype, vec, short_rows) : mx_quant_of<E2M1>(dtype, vec, short_rows);
}

// ------------------------------------------------------------------ a matrix's transpose

// A block of threads per tile of 128 rows x 64 columns (128 of 16-bit types), a thread per 32 rows
// of a column (of two neighbouring columns, loaded as one word where WORDS says that they are
// aligned), whose blocks of 32 of the transposed rows are its own: the loads run along the rows of
// x (lanes = columns).  The transposed rows go out through shared memory, 128 elements (64 code
// bytes) of a row at a time; a row's four scale bytes are one word.  Bound by memory: 6 x 2560 x 4096
// with values, fp32 83.5 us (537 MB, 6.4 TB/s), bf16 45.6 us (285 MB, 6.3 TB/s).
template <typename T, bool WORDS>
__global__ void __launch_bounds__(256) mx_quant_transposed_kernel(MxQuantArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kPer = 4 / (int)sizeof(T);           // columns of a thread
    constexpr int kCols = 64 * kPer;
    constexpr int kPitch = 128 + 16 / (int)sizeof(T);  // elements; 16-byte accesses of neighbouring
                                                       // columns fall into different banks
    extern __shared__ uint4 s_raw[];
    T* s_val = reinterpret_cast<T*>(s_raw);            // [kCols][kPitch]
    uint4* s_code = s_raw + kCols * kPitch * sizeof(T) / 16;  // [kCols][5]: 64 bytes, 16 of padding
    uint32_t* s_scale = reinterpret_cast<uint32_t*>(s_code + kCols * 5);  // [kCols]
    const int rt = div_up(a.rows, 128), ct = div_up(a.cols, kCols);
    const int blocks = a.rows >> 5;
    const int c = threadIdx.x % 64 * kPer, rq = threadIdx.x / 64;
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
            uint32_t e[32];  // an element, or two columns' elements
            const bool two = kPer == 2 && c + 1 < C;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                const T* p = x + q * a.row_stride;
                if constexpr (kPer == 1) {
                    e[q] = *reinterpret_cast<const uint32_t*>(p);
                } else if (WORDS && two) {
                    e[q] = *reinterpret_cast<const uint32_t*>(p);
                } else {
                    e[q] = *reinterpret_cast<const uint16_t*>(p);
                    if (two) e[q] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + 1) << 16;
                }
            }
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                if constexpr (kPer == 1) m = max(m, e[q] & 0x7FFFFFFFu);
                else m = Eight<T>::max_u16x2(m, e[q] & 0x7FFF7FFFu);
            }
#pragma unroll
            for (int h = 0; h < kPer; ++h) {
                if (c + h >= C) break;
                uint32_t am = m;
                if constexpr (kPer == 2) am = Eight<T>::bits16_f32(h ? m >> 16 : m & 0xFFFFu);
                const uint32_t s = mx_scale_byte<E2M1>(am, a.rule);
                const float scale = mx_encode_scale(s);
                uint32_t codes[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t w = e[8 * q + j];
                        v[j] = scale * __uint_as_float(
                                           kPer == 1 ? w : Eight<T>::bits16_f32(h ? w >> 16 : w & 0xFFFFu));
                    }
                    codes[q] = s == 255u ? 0u : f32x8_to_e2m1(v);
                }
                s_code[(c + h) * 5 + rq] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
                reinterpret_cast<uint8_t*>(&s_scale[c + h])[rq] = (uint8_t)s;
                if (a.values) {
                    const float d = mx_decode_scale(s);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float f[8];
                        e2m1x8_to_f32(codes[q], f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] *= d;
                        Eight<T> o;
                        o.from_f32(f);
                        o.store(s_val + (c + h) * kPitch + rq * 32 + 8 * q);
                    }
                }
            }
        }
        __syncthreads();
        const int64_t row0 = (b * a.cols + c0) * a.rows + tr * 128;  // element of column c0's row
        if (threadIdx.x < C)
            store_scales(a.sf, a.layout, b, a.cols, c0 + threadIdx.x, blocks, tr * 4, s_scale[threadIdx.x]);
        // codes: a thread per 16 bytes, four per column
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
            const int q = 64 * h + (threadIdx.x >> 2), p = threadIdx.x & 3;
            if (q < C && p * 32 < R)
                *reinterpret_cast<uint4*>(a.codes + (row0 + (int64_t)q * a.rows) / 2 + p * 16) = s_code[q * 5 + p];
        }
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

MxQuantKernel mx_quant_transposed_kernel_for(int dtype, bool words)
{
    switch (dtype) {
        case MOE_BF16:
            return words ? mx_quant_transposed_kernel<__nv_bfloat16, true> : mx_quant_transposed_kernel<__nv_bfloat16, false>;
        case MOE_FP16: return words ? mx_quant_transposed_kernel<__half, true> : mx_quant_transposed_kernel<__half, false>;
        default: return mx_quant_transposed_kernel<float, true>;
    }
}

// ------------------------------------------------------------------ scale layout

// A thread per 4-byte word of the tiled layout: four scales of one row, a byte at a time.  Runs once, when
// a checkpoint is loaded: 320 matrices of 2560 x 4096 (105 MB in, as much out) 344 us, 0.6 TB/s.
__global__ void __launch_bounds__(256) mx_tile_scales_kernel(const uint8_t* sf, int batch, int rows,
                                                             int blocks, uint8_t* tiled)
{
    const int RB = div_up(rows, 128), KA = (blocks + 3) >> 2;
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
