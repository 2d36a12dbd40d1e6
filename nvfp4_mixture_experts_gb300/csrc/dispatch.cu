// Tokens sorted by expert and back, with their gradients: the sort of the routed (token, expert)
// pairs, the row scatter (dispatch), the weighted row gather (combine, and dispatch's gradient)
// and combine's gradient.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.cuh"

namespace moe {

// ------------------------------------------------------------------ element types

// A piece of a row: V elements of type T in one access of B = V sizeof(T) bytes (16, 8, 4 or 2), the
// largest that every row of the call's tensors is aligned to.  fp32 values in, fp32 values out;
// rounding to nearest even.  (8192 rows of 4001 16-bit elements, aligned to nothing more, take 131
// us in combine where 4004, aligned to 8 bytes, take 90; reading 16-byte blocks around every piece
// and shifting them into place was measured at 167, and at 600 against 241 in combine's gradient:
// the blocks' registers cost more loads in flight than they save instructions.)
template <int B>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

template <typename T, int V>
struct Piece {
    typename Word<V * (int)sizeof(T)>::type raw;
    using W = decltype(raw);
    __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const W*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<W*>(p) = raw; }
    __device__ __forceinline__ void unpack(float (&f)[V]) const
    {
        if constexpr (V == 1) {
            T e;
            *reinterpret_cast<W*>(&e) = raw;
            f[0] = (float)e;
        } else {
            constexpr int N = V * (int)sizeof(T) / 4;
            alignas(16) uint32_t w[N];
            *reinterpret_cast<W*>(w) = raw;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if constexpr (sizeof(T) == 4) {
                    f[i] = __uint_as_float(w[i]);
                } else if constexpr (std::is_same<T, __half>::value) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    f[2 * i] = v.x;
                    f[2 * i + 1] = v.y;
                } else {
                    f[2 * i] = __uint_as_float(w[i] << 16);
                    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
            }
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[V])
    {
        if constexpr (V == 1) {
            T e;
            if constexpr (std::is_same<T, __half>::value) e = __float2half_rn(f[0]);
            else if constexpr (std::is_same<T, float>::value) e = f[0];
            else e = __float2bfloat16_rn(f[0]);
            raw = *reinterpret_cast<const W*>(&e);
        } else {
            constexpr int N = V * (int)sizeof(T) / 4;
            alignas(16) uint32_t w[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if constexpr (sizeof(T) == 4) {
                    w[i] = __float_as_uint(f[i]);
                } else if constexpr (std::is_same<T, __half>::value) {
                    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
            raw = *reinterpret_cast<const W*>(w);
        }
    }
};

// ------------------------------------------------------------------ the sort

// A stable counting sort.  Every warp that takes part owns a contiguous segment of the pairs and a
// table of counts by expert in shared memory.  Pass 1 counts the segments (32 pairs at a time:
// lanes of equal expert found with votes, their first lane adds their number, so no atomics).
// Prefix sums over the block's warps, over the blocks and over the experts (group sizes rounded up
// to row_align) turn the tables into the row of each segment's first pair of each expert.  Pass 2
// walks the segments again: a pair's row is its table entry plus the number of lower lanes of equal
// expert, and the first lane moves the entry on.
//
// Up to kSmallPairs pairs one block does it alone, in the launch that also moves the rows, every
// block of which sorts for itself (one token's dispatch 5.4 us so, 8.0 when the rows were moved by a
// second launch); more are shared out over the blocks of one thread block cluster, which read each
// other's totals through distributed shared memory.  A chain of latencies bounds both (loads, a dozen
// barriers, two cluster barriers): the maps of one token's 8 pairs over 320 experts take 3.9 us, over 8
// experts 2.5 (a launch that does nothing much 1.2), of 16384 pairs 6.5 us, 65536 pairs 10 us, 524288
// pairs 55 us.
struct SortShared {
    uint32_t tot[kMaxExperts];       // this block's pairs of each expert
    uint32_t off[kMaxExperts + 1];   // first row of each group
    uint32_t cnt[kMaxExperts];
    uint32_t warp[32];
};

__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* local, uint32_t rank)
{
    uint32_t v;
    asm volatile(
        "{\n\t.reg .b32 ra;\n\t"
        "mapa.shared::cluster.u32 ra, %1, %2;\n\t"
        "ld.shared::cluster.u32 %0, [ra];\n\t}"
        : "=r"(v)
        : "r"(smem_u32(local)), "r"(rank)
        : "memory");
    return v;
}

constexpr int kSortHold = 8;  // batches of 32 pairs that a warp keeps in registers between passes

// The lanes of the warp whose le (-1 .. El - 1) equals this lane's: one vote per bit of the
// numbers 0 .. El (a match instruction takes some 230 cycles on 32 different values, a vote a few).
__device__ __forceinline__ uint32_t equal_lanes(int le, int bits)
{
    const uint32_t key = (uint32_t)(le + 1);
    uint32_t same = 0xffffffffu;
    for (int i = 0; i < bits; ++i) {
        const bool set = (key >> i) & 1u;
        const uint32_t vote = __ballot_sync(0xffffffffu, set);
        same &= set ? vote : ~vote;
    }
    return same;
}

// Sorts with the `nw` first warps of each of `nblk` blocks (rank: this one's place).  calls
// emit(pair, row) for this block's pairs (row -1: dropped); leaves off and cnt in sh.  tab:
// [nw][El].  Ends with a block barrier for nblk 1; for more the caller ends with cluster_sync.
template <typename Emit>
__device__ __forceinline__ void sort_core(const SortArgs& a, SortShared& sh, uint32_t* tabs, int rank,
                                          int nblk, int nw, bool flag, Emit emit)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int El = a.El;
    uint32_t* tab = tabs + (size_t)warp * El;
    const bool works = warp < nw;
    const int64_t p0 = min((int64_t)a.P, ((int64_t)rank * nw + warp) * a.segment);
    const int64_t p1 = works ? min((int64_t)a.P, p0 + a.segment) : p0;
    auto local_expert = [&](int id, bool in, bool tell) {
        if (!in) return -1;
        if (id < 0 || id >= a.E) {
            if (tell) set_status(a.status, MOE_DEV_BAD_EXPERT_ID);
            return -1;
        }
        const int le = id - a.off;
        return (le >= 0 && le < El) ? le : -1;
    };
    int held[kSortHold];  // the first batches' ids, loaded together
#pragma unroll
    for (int i = 0; i < kSortHold; ++i) {
        const int64_t p = p0 + 32 * i + lane;
        held[i] = p < p1 ? a.ids[p] : 0;
    }
    if (works)
        for (int e = lane; e < El; e += 32) tab[e] = 0;
    __syncwarp();
    const int bits = 32 - __clz(El);
    auto count = [&](int le) {
        const uint32_t same = equal_lanes(le, bits);
        if (le >= 0 && lane == __ffs(same) - 1) tab[le] += __popc(same);
        __syncwarp();
        return same;
    };
    uint32_t same[kSortHold];
#pragma unroll
    for (int i = 0; i < kSortHold; ++i) {
        if (p0 + 32 * i >= p1) break;
        held[i] = local_expert(held[i], p0 + 32 * i + lane < p1, flag);
        same[i] = count(held[i]);
    }
    for (int64_t p = p0 + 32 * kSortHold; p < p1; p += 32)
        count(local_expert(p + lane < p1 ? a.ids[p + lane] : 0, p + lane < p1, flag));
    __syncthreads();
    // exclusive prefix over the block's warps, a thread per expert
    for (int e = tid; e < El; e += kSortThreads) {
        uint32_t run = 0;
#pragma unroll 8
        for (int w = 0; w < nw; ++w) {
            const uint32_t c = tabs[(size_t)w * El + e];
            tabs[(size_t)w * El + e] = run;
            run += c;
        }
        sh.tot[e] = run;
    }
    // pairs of each expert in the blocks before this one, and in all of them
    uint32_t before = 0, all = 0;
    if (nblk > 1) {
        cluster_sync();
        if (tid < El) {
            uint32_t c[kSortBlocks];
#pragma unroll
            for (int b = 0; b < kSortBlocks; ++b)
                c[b] = b >= nblk ? 0u : ld_cluster_u32(&sh.tot[tid], b);
#pragma unroll
            for (int b = 0; b < kSortBlocks; ++b) {
                if (b < rank) before += c[b];
                all += c[b];
            }
        }
    } else if (tid < El) {
        all = sh.tot[tid];
    }
    // first row of each group: exclusive scan of the counts rounded up
    const uint32_t padded = (all + a.align - 1) & ~(uint32_t)(a.align - 1);
    uint32_t x = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sh.warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        uint32_t v = sh.warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        sh.warp[lane] = v;
    }
    __syncthreads();
    const uint32_t first = x - padded + (warp ? sh.warp[warp - 1] : 0);
    if (tid < El) {
        sh.off[tid] = first;
        sh.cnt[tid] = all;
        if (tid == El - 1) sh.off[El] = first + padded;
#pragma unroll 8
        for (int w = 0; w < nw; ++w) tabs[(size_t)w * El + tid] += first + before;
    }
    if (El == 0 && tid == 0) sh.off[0] = 0;
    __syncthreads();
    auto place = [&](int64_t p, int le, uint32_t same) {
        int row = -1;
        if (le >= 0) {
            const uint32_t r = tab[le] + __popc(same & ((1u << lane) - 1u));
            if (r < (uint32_t)a.rows_cap) row = (int)r;
        }
        __syncwarp();
        if (le >= 0 && lane == __ffs(same) - 1) tab[le] += __popc(same);
        __syncwarp();
        if (p + lane < p1) emit((int32_t)(p + lane), row);
    };
#pragma unroll
    for (int i = 0; i < kSortHold; ++i) {
        if (p0 + 32 * i >= p1) break;
        place(p0 + 32 * i, held[i], same[i]);
    }
    for (int64_t p = p0 + 32 * kSortHold; p < p1; p += 32) {
        const bool in = p + lane < p1;
        const int le = local_expert(in ? a.ids[p + lane] : 0, in, false);
        place(p, le, equal_lanes(le, bits));
    }
}

// counts, offsets and the overflow flag (one block of the launch).
__device__ __forceinline__ void sort_write_groups(const SortArgs& a, const SortShared& sh)
{
    const int tid = threadIdx.x;
    for (int e = tid; e <= a.El; e += kSortThreads) a.offsets[e] = (int32_t)sh.off[e];
    for (int e = tid; e < a.El; e += kSortThreads) {
        a.counts[e] = (int32_t)sh.cnt[e];
        // rows past the capacity (padding alone may fall there)
        if (sh.cnt[e] && sh.off[e] + sh.cnt[e] > (uint32_t)a.rows_cap)
            set_status(a.status, MOE_DEV_ROWS_OVERFLOW);
    }
}

// perm_src of the rows of no pair, shared out over the launch's blocks.
__device__ __forceinline__ void sort_write_padding(const SortArgs& a, const SortShared& sh, int rank,
                                                   int nblk)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t cap = (uint32_t)a.rows_cap;
    for (int g = rank * 32 + warp; g < a.El; g += nblk * 32) {
        const uint32_t r1 = min(sh.off[g + 1], cap);
        for (uint32_t r = sh.off[g] + sh.cnt[g] + lane; r < r1; r += 32) a.perm_src[r] = -1;
    }
    for (uint32_t r = sh.off[a.El] + (uint32_t)rank * kSortThreads + tid; r < cap;
         r += (uint32_t)nblk * kSortThreads)
        a.perm_src[r] = -1;
}

__global__ void __launch_bounds__(kSortThreads) sort_pairs_kernel(SortArgs a)
{
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint32_t s_tab[];  // [32 warps][El]
    __shared__ SortShared sh;
    const int rank = blockIdx.x, nblk = gridDim.x;
    sort_core(a, sh, s_tab, rank, nblk, 32, true, [&](int32_t p, int row) {
        a.inv[p] = row;
        // scattered words, 32 sectors a warp: left to the kernel that moves the rows, where all
        // of the GPU shares them, if one follows
        if (row >= 0 && !a.rows_follow) a.perm_src[row] = p;
    });
    if (rank == 0) sort_write_groups(a, sh);
    sort_write_padding(a, sh, rank, nblk);
    if (nblk > 1) cluster_sync();  // no block leaves while another may read its totals
}

// The sort of up to kSmallPairs pairs and the rows' move (rows null: none) in one launch: every
// block sorts all pairs into shared memory and moves its share of the tokens.
template <typename U>
__global__ void __launch_bounds__(kSortThreads) dispatch_small_kernel(SortArgs a, DispatchArgs d)
{
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint32_t s_tab[];  // [warps that hold pairs][El]
    __shared__ SortShared sh;
    __shared__ int32_t s_row[kSmallPairs];
    const int rank = blockIdx.x, nblk = gridDim.x;
    sort_core(a, sh, s_tab, 0, 1, (a.P + 31) >> 5, rank == 0, [&](int32_t p, int row) {
        s_row[p] = row;
        if (rank == 0) {
            a.inv[p] = row;
            if (row >= 0) a.perm_src[row] = p;
        }
    });
    __syncthreads();
    if (d.rows) {
        const U* x = static_cast<const U*>(d.x);
        U* rows = static_cast<U*>(d.rows);
        for (int t = rank; t < d.T; t += nblk)
            for (int u = threadIdx.x; u < d.units; u += kSortThreads) {
                const U v = x[t * d.x_stride + u];
                for (int j = 0; j < d.k; ++j) {
                    const int row = s_row[t * d.k + j];
                    if (row >= 0) rows[(int64_t)row * d.units + u] = v;
                }
            }
    }
    if (rank == 0) sort_write_groups(a, sh);
    sort_write_padding(a, sh, rank, nblk);
}

DispatchSmallKernel dispatch_small_kernel_for(int unit_bytes)
{
    switch (unit_bytes) {
        case 16: return dispatch_small_kernel<uint4>;
        case 8: return dispatch_small_kernel<uint2>;
        case 4: return dispatch_small_kernel<uint32_t>;
        default: return dispatch_small_kernel<uint16_t>;
    }
}

// ------------------------------------------------------------------ dispatch

// rows[inv[t k + j]] = x[t]: a warp takes a run of pieces of one token and stores it to each of
// the token's rows, so x is read once.  Every warp loads its first run while the sort before it is
// still at work (x was complete before the sort began; 8192 tokens x 4096 bf16, k 8: 101 -> 98 us;
// prefetching the other runs into L2 meanwhile changed nothing: the writes are what takes the time).
// Rows of 4001 such elements, aligned to nothing more, move two bytes a lane: 123 us, eight times the
// loads and stores of the 98.
template <typename U>
__global__ void __launch_bounds__(256) dispatch_rows_kernel(DispatchArgs a)
{
    constexpr int kRun = kDispatchRun / 32;  // pieces per lane
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    const int runs = (a.units + 32 * kRun - 1) / (32 * kRun);
    const int64_t items = (int64_t)a.T * runs;
    const U* x = static_cast<const U*>(a.x);
    U* rows = static_cast<U*>(a.rows);
    U v[kRun];
    auto load = [&](int64_t i) {
        const int64_t t = i / runs;
        const int u0 = (int)(i - t * runs) * 32 * kRun + lane;
#pragma unroll
        for (int r = 0; r < kRun; ++r)
            if (u0 + 32 * r < a.units) v[r] = x[t * a.x_stride + u0 + 32 * r];
    };
    int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (i < items) load(i);
    pdl_wait();
    pdl_trigger();
    for (bool loaded = true; i < items; i += warps, loaded = false) {
        if (!loaded) load(i);
        const int64_t t = i / runs;
        const int u0 = (int)(i - t * runs) * 32 * kRun + lane;
        const bool full = u0 - lane + 32 * kRun <= a.units;
        for (int j = 0; j < a.k; ++j) {
            const int row = a.inv[t * a.k + j];
            if ((uint32_t)row >= (uint32_t)a.rows_cap) continue;
            if (u0 == 0) a.perm_src[row] = (int32_t)(t * a.k + j);
            U* to = rows + (int64_t)row * a.units + u0;
            if (full) {
#pragma unroll
                for (int r = 0; r < kRun; ++r) to[32 * r] = v[r];
            } else {
#pragma unroll
                for (int r = 0; r < kRun; ++r)
                    if (u0 + 32 * r < a.units) to[32 * r] = v[r];
            }
        }
    }
}

DispatchKernel dispatch_rows_kernel_for(int unit_bytes)
{
    switch (unit_bytes) {
        case 16: return dispatch_rows_kernel<uint4>;
        case 8: return dispatch_rows_kernel<uint2>;
        case 4: return dispatch_rows_kernel<uint32_t>;
        default: return dispatch_rows_kernel<uint16_t>;
    }
}

// ------------------------------------------------------------------ combine

// The pairs of a token: every lane of a warp holds one pair's row (-1 past k) and weight.
struct Pairs {
    int row;
    float w;
    __device__ __forceinline__ Pairs(const int32_t* inv, const float* weights, int64_t t, int k)
    {
        const int lane = threadIdx.x & 31;
        row = -1;
        w = 1.0f;
        if (lane < k) {
            row = inv[t * k + lane];
            if (weights) w = weights[t * k + lane];
        }
    }
    // the lanes of the kept pairs
    __device__ __forceinline__ uint32_t kept(int rows_cap) const
    {
        return __ballot_sync(0xffffffffu, (uint32_t)row < (uint32_t)rows_cap);
    }
};

// out[t] = sum_j w[t, j] rows[inv[t k + j]] (w null: 1): a warp takes a run of pieces of a token, the
// rows and weights of the token's pairs held by its lanes; dropped pairs cost nothing, of the kept
// ones four rows' loads are in flight at a time; fp32 sums in ascending j.  Bound by memory: 8192
// tokens x 4096 bf16, k 8: 91 us (604 MB, 6.6 TB/s); eight rows at a time need 115 registers, which
// halves the warps (92 us; 2048 x 4096 fp32 with half of the pairs kept 33 us, 27.5 with four).
template <typename T, int V>
__global__ void __launch_bounds__(256) combine_rows_kernel(CombineArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kPer = combine_run(V * (int)sizeof(T)) / 32, kAt = kCombineAt;
    const int lane = threadIdx.x & 31;
    const int units = a.H / V, runs = (units + 32 * kPer - 1) / (32 * kPer);
    const int64_t items = (int64_t)a.T * runs, step = (int64_t)gridDim.x * (blockDim.x >> 5);
    const T* y = static_cast<const T*>(a.y);
    T* out = static_cast<T*>(a.out);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < items; i += step) {
        const int64_t t = i / runs;
        const int u0 = (int)(i - t * runs) * 32 * kPer + lane;
        const bool full = u0 - lane + 32 * kPer <= units;
        const Pairs pairs(a.inv, a.w, t, a.k);
        float acc[kPer][V] = {};
        for (uint32_t kept = pairs.kept(a.rows_cap); kept;) {
            Piece<T, V> p[kAt][kPer];
            float w[kAt];
            const int n = min(__popc(kept), kAt);
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                if (j >= n) break;
                const int src = __ffs(kept) - 1;
                kept &= kept - 1;
                const int row = __shfl_sync(0xffffffffu, pairs.row, src);
                w[j] = __shfl_sync(0xffffffffu, pairs.w, src);
                const T* from = y + (int64_t)row * a.H + (int64_t)u0 * V;
                if (full) {
#pragma unroll
                    for (int q = 0; q < kPer; ++q) p[j][q].load(from + 32 * V * q);
                } else {
#pragma unroll
                    for (int q = 0; q < kPer; ++q)
                        if (u0 + 32 * q < units) p[j][q].load(from + 32 * V * q);
                }
            }
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                if (j >= n) break;
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    float f[V];
                    p[j][q].unpack(f);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[q][e] = fmaf(w[j], f[e], acc[q][e]);
                }
            }
        }
        T* to = out + t * a.out_stride + (int64_t)u0 * V;
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            if (full || u0 + 32 * q < units) {
                Piece<T, V> sum;
                sum.pack(acc[q]);
                sum.store(to + 32 * V * q);
            }
    }
}

// As combine_rows_kernel, for K pairs a token, one or two: a warp takes kCombineAt / K tokens at a time,
// so that as many rows' loads are in flight: 8192 tokens x 4096 bf16, k 1: 21.9 us (134 MB, 6.1 TB/s),
// k 2: 30.4 (201 MB, 6.6 TB/s).
template <typename T, int V, int K>
__global__ void __launch_bounds__(256) combine_few_kernel(CombineArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kPer = combine_run(V * (int)sizeof(T)) / 32, kTokens = kCombineAt / K;
    const int lane = threadIdx.x & 31;
    const int units = a.H / V, runs = (units + 32 * kPer - 1) / (32 * kPer);
    const int64_t items = (int64_t)div_up(a.T, kTokens) * runs;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
    const T* y = static_cast<const T*>(a.y);
    T* out = static_cast<T*>(a.out);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < items; i += step) {
        const int64_t b = i / runs, t0 = b * kTokens;
        const int u0 = (int)(i - b * runs) * 32 * kPer + lane;
        const int n = (int)min((int64_t)kTokens, a.T - t0);  // tokens
        int row = -1;
        float weight = 1.0f;
        if (lane < n * K) {
            row = a.inv[t0 * K + lane];
            if (a.w) weight = a.w[t0 * K + lane];
        }
        Piece<T, V> p[kCombineAt][kPer];
        bool kept[kCombineAt];
#pragma unroll
        for (int j = 0; j < kCombineAt; ++j) {
            const int r = __shfl_sync(0xffffffffu, row, j);
            kept[j] = (uint32_t)r < (uint32_t)a.rows_cap;
            if (!kept[j]) continue;
            const T* from = y + (int64_t)r * a.H + (int64_t)u0 * V;
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                if (u0 + 32 * q < units) p[j][q].load(from + 32 * V * q);
        }
#pragma unroll
        for (int m = 0; m < kTokens; ++m) {
            if (m >= n) break;
            T* to = out + (t0 + m) * a.out_stride + (int64_t)u0 * V;
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                float acc[V] = {};
#pragma unroll
                for (int j = m * K; j < (m + 1) * K; ++j) {
                    const float w = __shfl_sync(0xffffffffu, weight, j);
                    if (!kept[j]) continue;
                    float f[V];
                    p[j][q].unpack(f);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = fmaf(w, f[e], acc[e]);
                }
                if (u0 + 32 * q < units) {
                    Piece<T, V> sum;
                    sum.pack(acc);
                    sum.store(to + 32 * V * q);
                }
            }
        }
    }
}

template <typename T, int V>
static CombineKernel combine_rows_of(int few)
{
    return few == 1 ? combine_few_kernel<T, V, 1>
         : few == 2 ? combine_few_kernel<T, V, 2> : combine_rows_kernel<T, V>;
}

template <typename T>
static CombineKernel combine_rows_unit(int unit, int few)
{
    switch (unit / (int)sizeof(T)) {
        case 8: if constexpr (sizeof(T) == 2) return combine_rows_of<T, 8>(few);
        case 4: return combine_rows_of<T, 4>(few);
        case 2: return combine_rows_of<T, 2>(few);
        default: return combine_rows_of<T, 1>(few);
    }
}

CombineKernel combine_rows_kernel_for(int dtype, int unit, int few)
{
    switch (dtype) {
        case MOE_BF16: return combine_rows_unit<__nv_bfloat16>(unit, few);
        case MOE_FP16: return combine_rows_unit<__half>(unit, few);
        default: return combine_rows_unit<float>(unit, few);
    }
}

// ------------------------------------------------------------------ combine's gradient

// A block of W warps per token: dy rows = w dout, and the dot products <dout, y row> of the kept
// pairs, four rows at a time, reduced over the block: dout is read once for four rows, and dy leaves
// in the pass that reads y.  Bound by memory and, for short rows, by a token's chain of loads and
// sums: 8192 tokens x 2048 bf16, k 4: 47.5 us (302 MB, 6.4 TB/s); 7694 x 304, a quarter of six
// pairs kept: 8.3 us.
template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * W) combine_back_kernel(CombineBackArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kAt = kCombineAt, kPer = back_per(V * (int)sizeof(T));
    __shared__ float s_dot[2][W][kMaxTopK];  // of the even and the odd tokens of the block
    const int units = a.H / V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* dout = static_cast<const T*>(a.dout);
    const T* y = static_cast<const T*>(a.y);
    T* dy = static_cast<T*>(a.dy);
    int odd = 0;
    Pairs next(a.inv, a.w, blockIdx.x, a.k);  // (the grid has at most T blocks)
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, odd ^= 1) {
        const Pairs pairs = next;
        if (t + gridDim.x < a.T) next = Pairs(a.inv, a.w, t + gridDim.x, a.k);
        float sum = 0.0f;  // lane j: this warp's share of pair j's dot product
        for (uint32_t kept = pairs.kept(a.rows_cap); kept;) {
            const int n = min(__popc(kept), kAt);
            int row[kAt], src[kAt];
            float w[kAt], dot[kAt];
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                src[j] = j < n ? __ffs(kept) - 1 : 0;
                if (j < n) kept &= kept - 1;
                row[j] = __shfl_sync(0xffffffffu, pairs.row, src[j]);
                w[j] = __shfl_sync(0xffffffffu, pairs.w, src[j]);
                dot[j] = 0.0f;
            }
            for (int u0 = threadIdx.x; u0 < units; u0 += 32 * W * kPer) {
                const bool full = u0 - lane + 32 * W * (kPer - 1) + 31 < units;
                Piece<T, V> pd[kPer], p[kAt][kPer];
                const T* from = dout + t * a.dout_stride + (int64_t)u0 * V;
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (full || u0 + 32 * W * q < units) pd[q].load(from + 32 * W * V * q);
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < kAt; ++j) {
                        if (j >= n) break;
                        const T* yr = y + (int64_t)row[j] * a.H + (int64_t)u0 * V;
#pragma unroll
                        for (int q = 0; q < kPer; ++q)
                            if (full || u0 + 32 * W * q < units) p[j][q].load(yr + 32 * W * V * q);
                    }
                }
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    if (!full && u0 + 32 * W * q >= units) break;
                    float d[V];
                    pd[q].unpack(d);
#pragma unroll
                    for (int j = 0; j < kAt; ++j) {
                        if (j >= n) break;
                        if (a.dw) {
                            float f[V];
                            p[j][q].unpack(f);
#pragma unroll
                            for (int e = 0; e < V; ++e) dot[j] = fmaf(d[e], f[e], dot[j]);
                        }
                        if (dy) {
                            float g[V];
#pragma unroll
                            for (int e = 0; e < V; ++e) g[e] = w[j] * d[e];
                            Piece<T, V> pg;
                            pg.pack(g);
                            pg.store(dy + (int64_t)row[j] * a.H + (int64_t)(u0 + 32 * W * q) * V);
                        }
                    }
                }
            }
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < kAt; ++j) {
                    if (j >= n) break;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
                        dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
                    if (lane == src[j]) sum = dot[j];
                }
            }
        }
        if (a.dw) {
            if constexpr (W > 1) {
                if (lane < a.k) s_dot[odd][warp][lane] = sum;
                __syncthreads();  // (the other buffer is free again once every warp is here)
                if (warp == 0) {
                    sum = 0.0f;
                    if (lane < a.k)
                        for (int q = 0; q < W; ++q) sum += s_dot[odd][q][lane];
                }
            }
            if (warp == 0 && lane < a.k) a.dw[t * a.k + lane] = sum;
        }
    }
}

// As combine_back_kernel, for K pairs a token, one or two: kCombineAt / K tokens at a time, so that as many
// rows' loads are in flight: 8192 tokens x 4096 bf16, k 1: 36.8 us (201 MB, 5.5 TB/s), k 2: 52 (336 MB,
// 6.5 TB/s).
template <typename T, int V, int W, int K>
__global__ void __launch_bounds__(32 * W) combine_back_few_kernel(CombineBackArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kAt = kCombineAt, kPer = back_per(V * (int)sizeof(T)), kTokens = kAt / K;
    __shared__ float s_dot[2][W][kAt];  // of the even and the odd batches of the block
    const int units = a.H / V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* dout = static_cast<const T*>(a.dout);
    const T* y = static_cast<const T*>(a.y);
    T* dy = static_cast<T*>(a.dy);
    int odd = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < a.T; t0 += (int64_t)gridDim.x * kTokens, odd ^= 1) {
        const int n = (int)min((int64_t)kTokens, a.T - t0) * K;  // pairs
        int row = -1;
        float weight = 0.0f;
        if (lane < n) {
            row = a.inv[t0 * K + lane];
            weight = a.w[t0 * K + lane];
        }
        bool kept[kAt];
        float dot[kAt];
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
            kept[j] = (uint32_t)__shfl_sync(0xffffffffu, row, j) < (uint32_t)a.rows_cap;
            dot[j] = 0.0f;
        }
        for (int u = warp * 32; u < units; u += 32 * W * kPer) {  // (a warp's lanes stay together)
            const int u0 = u + lane;
            Piece<T, V> pd[kTokens][kPer], p[kAt][kPer];
#pragma unroll
            for (int m = 0; m < kTokens; ++m) {
                if (!kept[m * K] && !kept[m * K + K - 1]) continue;
                const T* from = dout + (t0 + m) * a.dout_stride + (int64_t)u0 * V;
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (u0 + 32 * W * q < units) pd[m][q].load(from + 32 * W * V * q);
            }
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < kAt; ++j) {
                    const int r = __shfl_sync(0xffffffffu, row, j);
                    if (!kept[j]) continue;
                    const T* yr = y + (int64_t)r * a.H + (int64_t)u0 * V;
#pragma unroll
                    for (int q = 0; q < kPer; ++q)
                        if (u0 + 32 * W * q < units) p[j][q].load(yr + 32 * W * V * q);
                }
            }
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                const int r = __shfl_sync(0xffffffffu, row, j);
                const float w = __shfl_sync(0xffffffffu, weight, j);
                if (!kept[j]) continue;
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    if (u0 + 32 * W * q >= units) break;
                    float d[V];
                    pd[j / K][q].unpack(d);
                    if (a.dw) {
                        float f[V];
                        p[j][q].unpack(f);
#pragma unroll
                        for (int e = 0; e < V; ++e) dot[j] = fmaf(d[e], f[e], dot[j]);
                    }
                    if (dy) {
                        float g[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) g[e] = w * d[e];
                        Piece<T, V> pg;
                        pg.pack(g);
                        pg.store(dy + (int64_t)r * a.H + (int64_t)(u0 + 32 * W * q) * V);
                    }
                }
            }
        }
        if (a.dw) {
            float sum = 0.0f;  // lane j: this warp's share of pair j's dot product
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
                if (lane == j) sum = dot[j];
            }
            if constexpr (W > 1) {
                if (lane < n) s_dot[odd][warp][lane] = sum;
                __syncthreads();  // (the other buffer is free again once every warp is here)
                if (warp == 0) {
                    sum = 0.0f;
                    if (lane < n)
                        for (int q = 0; q < W; ++q) sum += s_dot[odd][q][lane];
                }
            }
            if (warp == 0 && lane < n) a.dw[t0 * K + lane] = sum;
        }
    }
}

// As combine_back_kernel, for long rows and more than four pairs a token: eight pairs at a time,
// kept or not, their rows and weights loaded by every thread alike (addresses in uniform registers),
// so that dout is read once.  Bound by memory: 8192 tokens x 4096 bf16, k 8: 169.5 us (1.14 GB, 6.7
// TB/s).
template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * W) combine_back_all_kernel(CombineBackArgs a)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float s_dot[W][8];
    const int units = a.H / V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* dout = static_cast<const T*>(a.dout);
    const T* y = static_cast<const T*>(a.y);
    T* dy = static_cast<T*>(a.dy);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        for (int j0 = 0; j0 < a.k; j0 += 8) {
            int row[8];
            float w[8], dot[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dot[j] = 0.0f;
                w[j] = 0.0f;
                row[j] = -1;
                if (j0 + j < a.k) {
                    const int r = a.inv[t * a.k + j0 + j];
                    if ((uint32_t)r < (uint32_t)a.rows_cap) {
                        row[j] = r;
                        w[j] = a.w[t * a.k + j0 + j];
                    }
                }
            }
            constexpr int kPer = back_per(V * (int)sizeof(T));  // pieces of a row in flight
            for (int u0 = threadIdx.x; u0 < units; u0 += 32 * W * kPer) {
                const bool full = u0 - lane + 32 * W * (kPer - 1) + 31 < units;
                Piece<T, V> pd[kPer], p[8][kPer];
                const T* from = dout + t * a.dout_stride + (int64_t)u0 * V;
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (full || u0 + 32 * W * q < units) pd[q].load(from + 32 * W * V * q);
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (row[j] >= 0) {
                            const T* yr = y + (int64_t)row[j] * a.H + (int64_t)u0 * V;
#pragma unroll
                            for (int q = 0; q < kPer; ++q)
                                if (full || u0 + 32 * W * q < units) p[j][q].load(yr + 32 * W * V * q);
                        }
                }
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    if (!full && u0 + 32 * W * q >= units) break;
                    float d[V];
                    pd[q].unpack(d);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (row[j] < 0) continue;
                        if (a.dw) {
                            float f[V];
                            p[j][q].unpack(f);
#pragma unroll
                            for (int e = 0; e < V; ++e) dot[j] = fmaf(d[e], f[e], dot[j]);
                        }
                        if (dy) {
                            float g[V];
#pragma unroll
                            for (int e = 0; e < V; ++e) g[e] = w[j] * d[e];
                            Piece<T, V> pg;
                            pg.pack(g);
                            pg.store(dy + (int64_t)row[j] * a.H + (int64_t)(u0 + 32 * W * q) * V);
                        }
                    }
                }
            }
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
                        dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
                    if (lane == 0) s_dot[warp][j] = dot[j];
                }
                __syncthreads();
                if (threadIdx.x < 8 && j0 + (int)threadIdx.x < a.k) {
                    float sum = 0.0f;
                    for (int q = 0; q < W; ++q) sum += s_dot[q][threadIdx.x];
                    a.dw[t * a.k + j0 + threadIdx.x] = sum;
                }
                __syncthreads();
            }
        }
    }
}

template <typename T, int V, int W>
static CombineBackKernel combine_back_warps(int few, bool all)
{
    if (few == 1) return combine_back_few_kernel<T, V, W, 1>;
    if (few == 2) return combine_back_few_kernel<T, V, W, 2>;
    if constexpr (W > 1) {
        if (all) return combine_back_all_kernel<T, V, W>;
    }
    return combine_back_kernel<T, V, W>;
}

template <typename T, int V>
static CombineBackKernel combine_back_of(int warps, int few, bool all)
{
    switch (warps) {
        case 1: return combine_back_warps<T, V, 1>(few, all);
        case 2: return combine_back_warps<T, V, 2>(few, all);
        case 4: return combine_back_warps<T, V, 4>(few, all);
        default: return combine_back_warps<T, V, 8>(few, all);
    }
}

template <typename T>
static CombineBackKernel combine_back_unit(int unit, int warps, int few, bool all)
{
    switch (unit / (int)sizeof(T)) {
        case 8: if constexpr (sizeof(T) == 2) return combine_back_of<T, 8>(warps, few, all);
        case 4: return combine_back_of<T, 4>(warps, few, all);
        case 2: return combine_back_of<T, 2>(warps, few, all);
        default: return combine_back_of<T, 1>(warps, few, all);
    }
}

CombineBackKernel combine_back_kernel_for(int dtype, int unit, int warps, int few, bool all)
{
    switch (dtype) {
        case MOE_BF16: return combine_back_unit<__nv_bfloat16>(unit, warps, few, all);
        case MOE_FP16: return combine_back_unit<__half>(unit, warps, few, all);
        default: return combine_back_unit<float>(unit, warps, few, all);
    }
}

}  // namespace moe
