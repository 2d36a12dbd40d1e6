// The grouped MXFP4 product on CTA pairs: out[r][n] = sum_i A[r][i] W_g[n][i] over the rows r of
// each group g.
//
// One tile is 256 weight rows (the MMA's M side: 128 in each CTA of the pair) by up to 256 rows of
// one group (its N side, in steps of 32: a group costs round_up(rows, 32) columns, where rows on
// the M side would cost a multiple of 128), the whole contraction in order, so nothing is summed
// across tiles and results do not depend on the schedule.  tcgen05.mma.cta_group::2 with
// kind::mxf4 multiplies E2M1 operands from shared memory under UE8M0 scales (one per 32 elements)
// from TMEM.  Each CTA loads its own 128 weight rows and half of the group's rows, so a
// 256-element k-stage brings 35 KB through each SM for 128 x 256 x 256 multiply-adds, where a CTA
// by itself would need 51 KB.
//
// Warp roles (both CTAs unless said): warp 0 issues the TMA loads of its CTA's operands and
// scales, all counted on the leader's stage barrier; warp 1 of the leader (cluster rank 0) copies
// each stage's scales to TMEM (tcgen05.cp, in order with the MMAs) and issues the MMAs; warps
// 2..9 read the accumulator (lane = weight row, column = group row) into registers, which frees it
// for the MMAs, transpose it through shared memory and store whole 128-column rows.
//
// What bounds it.  Memory where weights are read once: 8192 tokens of 320 experts, N 2560, K 4096,
// 326 us for 2.26 GB (6.9 TB/s, 4.2 PFLOP/s); 64 tokens, 198 us (7.1 TB/s); 257 tokens on 160
// experts, N 4096, K 1280, fp32 out, 67.6 us (6.8 TB/s).  With few rows and few tiles the two
// threads that issue loads and MMAs, 0.18 us a k-stage: one row, N 4096, K 4096 6.7 us, K 16384
// 15.6 us (4 us of launch, group table, epilogue and exit); the last tiles of one token's gate_up
// over 320 experts (80 tiles for 76 pairs) take 3 of its 12 us so.  With many rows the tensor pipe
// (four MMAs 0.26 us a k-stage, 0.28 where 16 pairs work: 256 rows, N 4096, K 16384 23 us) and, where
// all pairs do, by its figures L2: 36 KB per SM and k-stage in 0.38 us, 14 TB/s (one group of 8192,
// N and K 4096: 46 us, 5.9 PFLOP/s, 0.69 of the tensor pipe).
//
// No tile is split along its contraction, also where there are fewer tiles than pairs: the parts
// would have to be written, counted and added up, through words that are zero before the call or
// CTAs that wait for one another, for 2 us at most.  Fetching the last tiles' weights into L2 during
// the tiles before gains nothing (13.9 us where 13.4 without).
//
// TMEM (all 512 columns, so the allocation starts at column 0): two accumulators, of the even
// tiles at column 0 upwards, of the odd tiles ending at column 448; two slots of a stage's scales
// in columns 448..511.  Two tiles of together up to 448 columns overlap freely: the next tile's
// MMAs run while one is read out.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kAccEnd = 448;                 // TMEM columns of accumulators; scales above
constexpr uint64_t kCopyLandNs = 1000000;    // after a wait that ran out, for copies in flight

struct Ctl {
    uint64_t full[kMxMaxStages], empty[kMxMaxStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort_flag, zero;
};
static_assert(sizeof(Ctl) <= kMxCtlBytes, "control block");

// One lane of a converged warp, the same one each time: the compiler knows that code under it runs
// in one thread, so the operands of the TMA and tcgen05 instructions stay in uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Tensor loads of a CTA pair: the bytes may be counted on the barrier of either CTA (bar is a
// shared::cluster address).
__device__ __forceinline__ void tma_pair_2d(void* dst, const CUtensorMap* m, uint32_t bar,
                                            int32_t x, int32_t y, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_pair_3d(void* dst, const CUtensorMap* m, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

// One 512-byte scale atom of each CTA's shared memory into its own TMEM (as tc_cp_sf, for a pair).
__device__ __forceinline__ void tc_cp_sf_pair(uint32_t taddr, uint64_t sdesc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
                 : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 x E2M1, UE8M0 scales, fp32 accumulation, both
// operands K-major; the scale ids (which two of the four bytes of a scale column a K = 64 step
// uses) are added per step.
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N)
{
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 7) << 27);
}

__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d_taddr, uint64_t adesc, uint64_t bdesc,
                                                 uint32_t idesc, uint32_t sfa_taddr,
                                                 uint32_t sfb_taddr, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_taddr),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_taddr), "r"(sfb_taddr), "r"(accumulate)
        : "memory");
}

// What a tile covers.  Tiles run over the groups' token tiles (256 group rows), and inside one
// over the 256-row weight tiles, so that tiles in flight at a time share their group rows in L2.
struct Tile {
    int g, n0;       // group; first weight row
    int rows, row0;  // group rows of the tile (1..256); first row of the tile in A
    int nt;          // columns of the MMA: rows rounded up to 32
};

struct Groups {
    const int32_t* start;   // [G + 1] first token tile of each group
    const int32_t* counts;  // [G] rows (0 for a skipped group)
    const int32_t* first;   // [G] first row
    int G, NB;
    int most;               // rows of the largest group
};

// The tile of index t (all lanes of a warp).  Its group, the last one that starts at or before the
// token tile, is found in two votes: the 32 groups it is among, then the one.
__device__ __forceinline__ Tile find_tile(const Groups& gs, int t)
{
    const int lane = threadIdx.x & 31;
    const int tt = t / gs.NB;
    const int c = lane * 32;
    const int coarse = (__popc(__ballot_sync(0xffffffffu, c < gs.G && gs.start[c] <= tt)) - 1) * 32;
    const int f = coarse + lane;
    const int g = coarse + __popc(__ballot_sync(0xffffffffu, f < gs.G && gs.start[f] <= tt)) - 1;
    Tile ti;
    ti.g = g;
    ti.n0 = (t - tt * gs.NB) * 256;
    const int r = (tt - gs.start[g]) * kMxTileRows;
    ti.rows = min(kMxTileRows, gs.counts[g] - r);
    ti.row0 = gs.first[g] + r;
    ti.nt = (ti.rows + 31) & ~31;
    return ti;
}

// Token tiles of the groups and their exclusive prefix, in shared memory (all threads; ends with
// __syncthreads).  A group whose rows do not start on a multiple of 128 or leave the capacity is
// flagged and gets none.
__device__ __forceinline__ Groups load_groups(const MxGemmArgs& a, int32_t* sm, int32_t* s_warp)
{
    constexpr int kPer = (kMaxExperts + kMxThreads - 1) / kMxThreads;  // groups of a thread at most
    const int G = a.G, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t* start = sm;
    int32_t* cnt = start + G + 1;
    int32_t* first = cnt + G;
    const int per = (G + kMxThreads - 1) / kMxThreads, g0 = tid * per;
    int c[kPer], o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool in = i < per && g0 + i < G;
        c[i] = !in ? 0 : a.counts ? a.counts[g0 + i] : a.rows_cap;
        o[i] = in && a.offsets ? a.offsets[g0 + i] : 0;
    }
    int sum = 0, most = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (c[i] > 0 && (o[i] < 0 || (o[i] & 127) || (int64_t)o[i] + c[i] > a.rows_cap)) {
            set_status(a.status, MOE_DEV_BAD_INDEX);
            c[i] = 0;
        }
        c[i] = max(c[i], 0);
        most = max(most, c[i]);
        sum += div_up(c[i], kMxTileRows);
    }
    int v = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += y;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) s_warp[warp] = v;
    if (lane == 0) s_warp[32 + warp] = most;
    __syncthreads();
    constexpr int kWarps = kMxThreads / 32;
    int pre = v - sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) pre += s_warp[w];
        most = max(most, s_warp[32 + w]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i < per && g0 + i < G) {
            start[g0 + i] = pre;
            cnt[g0 + i] = c[i];
            first[g0 + i] = o[i];
            pre += div_up(c[i], kMxTileRows);
        }
    if (tid == kMxThreads - 1) start[G] = pre;  // (no groups of its own, or the last ones)
    __syncthreads();
    return Groups{start, cnt, first, G, div_up(a.N, 256), most};
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns = kWaitLimitNs)
{
    int ok = 1;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort, limit_ns) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The ring of k-stages in shared memory.  Where no group has more than 64 rows a stage holds 32
// group rows per CTA and one row block of scales instead of 128 and two, and nine of them fit
// instead of six (one token's gate_up with five stages of the large kind: 16.3 us, so 13.8).
struct Stages {
    uint8_t* base;
    int n;                                   // stages
    uint32_t bytes, t, sw, st;               // of a stage; offsets of its parts (weights at 0)
    __device__ __forceinline__ Stages(uint8_t* p, int big, bool small) : base(p)
    {
        n = small ? big * kMxStageBytes / kMxSmallStageBytes : big;
        bytes = small ? kMxSmallStageBytes : kMxStageBytes;
        t = 16384;
        sw = t + (small ? 4096 : 16384);
        st = sw + 1024;
    }
};

struct Place {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++stage == n) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// Each thread of the warp reads 2 x 16 lanes x 32 columns of TMEM from taddr: register 4 i + e of
// half h holds lane 16 h + l / 4 + 8 (e / 2), column 8 i + 2 (l % 4) + e % 2 (l: the thread's lane).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[32])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t* q = r + 16 * h;
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]),
              "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]),
              "=r"(q[13]), "=r"(q[14]), "=r"(q[15])
            : "r"(taddr + ((uint32_t)(16 * h) << 16))
            : "memory");
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A chunk of the accumulator: 32 weight rows (TMEM lanes) x 32 group rows (columns).
template <typename T>
__device__ __forceinline__ void load_chunk(uint32_t taddr, uint32_t (&r)[32])
{
    if constexpr (sizeof(T) == 2) tmem_ld_frag(taddr, r);
    else tmem_ld32(taddr, r);
}

// A barrier of the four epilogue warps of a group.
__device__ __forceinline__ void group_sync(int group)
{
    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// The same, and whether all four warps say ok: of four waits for one phase, some may see it complete
// and others run out, and a warp that left alone would leave the rest at their next barrier.
__device__ __forceinline__ bool group_all(int group, bool ok)
{
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)ok), "r"(1 + group)
        : "memory");
    return all != 0;
}

// Stores a group's staged rows j0 .. j0 + ROWS - 1 (of `live`): columns n0 .. n0 + 127 in pieces of
// type U, the largest (16, 4 or, 16-bit types, 2 bytes) that every output row is aligned to and a
// whole number of; th: the thread of the group.
template <typename T, typename U, int ROWS, int PITCH>
__device__ __forceinline__ void store_rows(const MxGemmArgs& a, const uint8_t* stage, T* out, int j0,
                                           int live, int n0, int th)
{
    constexpr int kPer = (int)sizeof(U) / (int)sizeof(T);  // elements of a piece
    constexpr int kLanes = 128 / kPer;                     // pieces of a row
    constexpr int kAt = 128 / kLanes;                      // rows at a time
    const int n = n0 + (th % kLanes) * kPer, jl = th / kLanes;
    if (n >= a.N) return;
    T* o = out + (int64_t)(j0 + jl) * a.out_stride + n;
    const uint8_t* st = stage + jl * PITCH + (th % kLanes) * (int)sizeof(U);
    U v[ROWS / kAt];
#pragma unroll
    for (int j = 0; j < ROWS / kAt; ++j) v[j] = *reinterpret_cast<const U*>(st + j * kAt * PITCH);
#pragma unroll
    for (int j = 0; j < ROWS / kAt; ++j)
        if (j0 + j * kAt + jl < live) *reinterpret_cast<U*>(o + (int64_t)(j * kAt) * a.out_stride) = v[j];
}

// Stores the chunks of a group's four warps: columns n0 .. n0 + 127 (this warp holds the 32 from
// 32 q) of the `live` first of 32 rows, out pointing at the first row.  A few rows at a time the
// chunks are transposed into the group's staging buffer (16-bit types: 8 x 8 matrices stored
// transposed; fp32: a word per lane and row) and leave as 16-byte pieces of whole 128-column rows
// (256 or 512 contiguous bytes), or in the smaller pieces that the output's rows are aligned to.  free:
// the group has passed a barrier since it last read the buffer.
template <typename T>
__device__ __forceinline__ void store_chunk(const MxGemmArgs& a, const uint32_t (&r)[32],
                                            uint8_t* stage, T* out, int live, int n0, int q,
                                            int group, int lane, bool free)
{
    constexpr int kPitch = mx_epi_pitch((int)sizeof(T));  // bytes of a staged row
    constexpr int kRows = mx_epi_rows((int)sizeof(T));    // rows staged at a time
#pragma unroll
    for (int j0 = 0; j0 < 32; j0 += kRows) {
        if (j0 >= live) break;
        if (j0 || !free) group_sync(group);  // the buffer has been read
        if constexpr (sizeof(T) == 2) {
            const uint32_t at = smem_u32(stage) + (lane & 7) * kPitch + q * 64 + (lane >> 3) * 16;
#pragma unroll
            for (int i = j0 / 8; i < (j0 + kRows) / 8; ++i) {
                uint32_t m[4];  // features 8 m .. 8 m + 7 of rows 8 i .. 8 i + 7
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int e = 16 * (f >> 1) + 4 * i + 2 * (f & 1);
                    m[f] = pack2(__uint_as_float(r[e]), __uint_as_float(r[e + 1]), T());
                }
                asm volatile(
                    "stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                        at + (8 * i - j0) * kPitch),
                    "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3])
                    : "memory");
            }
        } else {
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                *reinterpret_cast<uint32_t*>(stage + j * kPitch + 4 * (32 * q + lane)) = r[j0 + j];
        }
        group_sync(group);
        const int th = 32 * q + lane;  // thread of the group
        if (a.unit == 16) {
            store_rows<T, uint4, kRows, kPitch>(a, stage, out, j0, live, n0, th);
        } else if (a.unit == 4) {
            store_rows<T, uint32_t, kRows, kPitch>(a, stage, out, j0, live, n0, th);
        } else if constexpr (sizeof(T) == 2) {
            store_rows<T, uint16_t, kRows, kPitch>(a, stage, out, j0, live, n0, th);
        }
    }
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kMxThreads, 1)
    gemm_mxfp4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
                      const __grid_constant__ CUtensorMap tmT16,
                      const __grid_constant__ CUtensorMap tmSW,
                      const __grid_constant__ CUtensorMap tmST, MxGemmArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    uint8_t* staging = ring + args.stages * kMxStageBytes;
    Ctl& ctl = *reinterpret_cast<Ctl*>(staging + mx_epi_bytes((int)sizeof(T)));
    int32_t* tables = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(&ctl) + kMxCtlBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int KB = div_up(args.K, 256);

    if (warp == 0 && elect_one()) {
        for (int s = 0; s < kMxMaxStages; ++s) {
            mbar_init(&ctl.full[s], 1);
            mbar_init(&ctl.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl.acc_full[b], 1);
            mbar_init(&ctl.acc_empty[b], 2 * kMxEpiWarps);  // both CTAs' (the leader's barrier)
        }
        mbar_init(&ctl.drain, 1);
        ctl.abort_flag = ctl.zero = 0;
        fence_barrier_init();
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmT);
        prefetch_tmap(&tmT16);
        prefetch_tmap(&tmSW);
        prefetch_tmap(&tmST);
    }
    __syncwarp();
    if (warp == 1) tmem_alloc_pair(&ctl.tmem, 512);
    tc_fence_before();
    // Group rows are read by every weight tile: kept in L2 (evicted first instead: 8192 tokens'
    // gate_up 332 -> 402 us).  Weights pass once where groups have few rows (evicted first: 64
    // tokens' gate_up 206 -> 201 us), but elsewhere neighbouring 128-byte pieces of their rows, which
    // L2 fetches in pairs, must outlive a k-stage (normal: 8192 tokens' down 244 -> 226 us).
    const uint64_t pol_first = policy_evict_first(), pol_normal = policy_evict_normal();
    const uint64_t pol_t = policy_evict_last();
    cluster_arrive();  // this CTA's barriers exist and its TMEM is allocated
    pdl_wait();
    pdl_trigger();
    const Groups gs = load_groups(args, tables, reinterpret_cast<int32_t*>(staging));
    cluster_wait();    // ... and the peer's
    tc_fence_after();
    const int ntiles = gs.start[gs.G] * gs.NB;
    const Stages sg(ring, args.stages, gs.most <= 64);
    volatile int* abort = &ctl.abort_flag;

    if (warp == 0) {
        const uint64_t pol_w = gs.most <= 64 ? pol_first : pol_normal;
        const uint32_t full0 = cluster_addr(&ctl.full[0], 0);  // the leader's barriers
        Place at;               // (the elected lane's)
        int issued = 0;         // stages with a copy of this CTA, the last one before `at`
        bool ok = true;
        for (int t = pair; t < ntiles && ok; t += npairs) {
            const Tile ti = find_tile(gs, t);
            if (elect_one()) {
                const int half = ti.nt >> 1;                    // group rows of this CTA
                const int trow = ti.row0 + (int)rank * half, wrow = ti.n0 + (int)rank * 128;
                const int nsc = ti.nt > 128 ? 2 : 1;            // row blocks of group-row scales
                const uint32_t bytes = 2u * (16384 + 1024 + half * 128 + nsc * 1024);
                const int wb = ti.g * div_up(args.N, 128) + (wrow >> 7), tb = ti.row0 >> 7;
                // A loop of its own for few rows, where this thread is what a lone tile waits for
                // (one row, N 4096, K 16384: 18.2 us in the other loop, 16.7 in this one).
                int kb = 0;
                if (half == 16) {
                    for (; kb < KB; ++kb) {
                        if (!mbar_wait(&ctl.empty[at.stage], at.phase ^ 1u, abort)) break;
                        uint8_t* p = sg.base + at.stage * sg.bytes;
                        const uint32_t bar = full0 + at.stage * 8;
                        if (rank == 0) mbar_arrive_expect_tx(&ctl.full[at.stage], bytes);
                        tma_pair_3d(p, &tmW, bar, kb * 32, wrow, ti.g, pol_w);
                        tma_pair_2d(p + sg.sw, &tmSW, bar, kb * 256, wb, pol_w);
                        tma_pair_2d(p + sg.t, &tmT16, bar, kb * 32, trow, pol_t);
                        tma_pair_2d(p + sg.st, &tmST, bar, kb * 256, tb, pol_t);
                        at.next(sg.n);
                    }
                } else {
                    for (; kb < KB; ++kb) {
                        if (!mbar_wait(&ctl.empty[at.stage], at.phase ^ 1u, abort)) break;
                        uint8_t* p = sg.base + at.stage * sg.bytes;
                        const uint32_t bar = full0 + at.stage * 8;
                        if (rank == 0) mbar_arrive_expect_tx(&ctl.full[at.stage], bytes);
                        tma_pair_3d(p, &tmW, bar, kb * 32, wrow, ti.g, pol_w);
                        tma_pair_2d(p + sg.sw, &tmSW, bar, kb * 256, wb, pol_w);
                        if (half == 128) {
                            tma_pair_2d(p + sg.t, &tmT, bar, kb * 32, trow, pol_t);
                        } else {
                            for (int i = 0; i < half; i += 16)
                                tma_pair_2d(p + sg.t + i * 128, &tmT16, bar, kb * 32, trow + i, pol_t);
                        }
                        tma_pair_2d(p + sg.st, &tmST, bar, kb * 256, tb, pol_t);
                        if (nsc == 2) tma_pair_2d(p + sg.st + 1024, &tmST, bar, kb * 256, tb + 1, pol_t);
                        at.next(sg.n);
                    }
                }
                issued = min(issued + kb, sg.n);
                ok = kb == KB;
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        if (elect_one()) {
            if (!ok) {
                set_status(args.status, MOE_DEV_WAIT_TIMEOUT);
                *abort = 1;
            }
            if (rank == 0)  // both CTAs' copies in flight land before either exits
                for (; issued > 0; --issued) {
                    if (--at.stage < 0) {
                        at.stage = sg.n - 1;
                        at.phase ^= 1u;
                    }
                    mbar_wait(&ctl.full[at.stage], at.phase, &ctl.zero);
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t s0 = smem_u32(sg.base);
            const uint64_t w0 = sdesc_sw128(s0), t0 = sdesc_sw128(s0 + sg.t);
            const uint64_t cw0 = sdesc_sf(s0 + sg.sw), ct0 = sdesc_sf(s0 + sg.st);
            int it = 0, prev_nt = 0;
            uint32_t slot = 0;
            Place at;  // (the elected lane's)
            bool ok = true;
            for (int t = pair; t < ntiles && ok; t += npairs, ++it) {
                const Tile ti = find_tile(gs, t);
                if (elect_one()) {
                    const int buf = it & 1;
                    // the accumulator's last user has been read out; so has the previous tile's
                    // where the two overlap
                    ok = mbar_wait_cluster(&ctl.acc_empty[buf], ((it >> 1) & 1) ^ 1u, abort);
                    if (ok && it && ti.nt + prev_nt > kAccEnd)
                        ok = mbar_wait_cluster(&ctl.acc_empty[buf ^ 1], ((it - 1) >> 1) & 1, abort);
                    tc_fence_after();
                    const uint32_t d_t = buf ? kAccEnd - ti.nt : 0;
                    const uint32_t idesc = idesc_mxf4(256, ti.nt), idesc2 = idesc | (2u << 4) | (2u << 29);
                    const bool two = ti.nt > 128;  // row blocks of group-row scales
                    // a stage's barrier is looked at before the MMAs of the one before are issued
                    // (one row, N 4096, K 16384: 16.7 us without, 15.6 with)
                    bool ready = mbar_test(&ctl.full[at.stage], at.phase);
                    for (int kb = 0; kb < KB && ok; ++kb) {
                        ok = ready || mbar_wait(&ctl.full[at.stage], at.phase, abort);
                        if (!ok) break;
                        tc_fence_after();
                        Place next = at;
                        next.next(sg.n);
                        ready = mbar_test(&ctl.full[next.stage], next.phase);
                        const uint32_t o = at.stage * (sg.bytes >> 4);  // descriptor units
                        const uint64_t w = w0 + o, tk = t0 + o, cw = cw0 + o, ct = ct0 + o;
                        const uint32_t sc = kAccEnd + slot;
                        const int left = args.K - kb * 256;
                        if (left >= 256) {
                            tc_cp_sf_pair(sc, cw);
                            tc_cp_sf_pair(sc + 8, ct);
                            if (two) tc_cp_sf_pair(sc + 12, ct + 64);
                            tc_cp_sf_pair(sc + 4, cw + 32);
                            tc_cp_sf_pair(sc + 16, ct + 32);
                            if (two) tc_cp_sf_pair(sc + 20, ct + 96);
                            tc_mma_mxf4_pair(d_t, w, tk, idesc, sc, sc + 8, kb != 0);
                            tc_mma_mxf4_pair(d_t, w + 2, tk + 2, idesc2, sc, sc + 8, 1);
                            tc_mma_mxf4_pair(d_t, w + 4, tk + 4, idesc, sc + 4, sc + 16, 1);
                            tc_mma_mxf4_pair(d_t, w + 6, tk + 6, idesc2, sc + 4, sc + 16, 1);
                        } else {  // the last k-stage: K = 64 steps that hold any of it
                            for (int j = 0; 64 * j < left; ++j) {
                                const int ka = j >> 1;
                                if (!(j & 1)) {
                                    tc_cp_sf_pair(sc + 4 * ka, cw + 32 * ka);
                                    tc_cp_sf_pair(sc + 8 + 8 * ka, ct + 32 * ka);
                                    if (two) tc_cp_sf_pair(sc + 12 + 8 * ka, ct + 64 + 32 * ka);
                                }
                                tc_mma_mxf4_pair(d_t, w + 2 * j, tk + 2 * j, (j & 1) ? idesc2 : idesc,
                                                 sc + 4 * ka, sc + 8 + 8 * ka, (kb | j) != 0);
                            }
                        }
                        tc_commit_pair(&ctl.empty[at.stage], 3);
                        slot ^= 32u;
                        at = next;
                    }
                    if (ok) tc_commit_pair(&ctl.acc_full[buf], 3);
                }
                prev_nt = ti.nt;
                ok = __all_sync(0xffffffffu, ok);
            }
            if (elect_one()) {  // the thread that issued the MMAs
                if (!ok) {
                    set_status(args.status, MOE_DEV_WAIT_TIMEOUT);
                    *abort = 1;
                }
                tc_commit_pair(&ctl.drain, 1);  // every MMA issued above is complete after this
                mbar_wait(&ctl.drain, 0, &ctl.zero);
            }
            __syncwarp();
        }
    } else {
        const int q = warp & 3, h = (warp - 2) >> 2;  // TMEM lane quarter; which 32-row chunks
        uint8_t* stage = staging + h * (mx_epi_bytes((int)sizeof(T)) / 2);
        int it = 0;
        for (int t = pair; t < ntiles; t += npairs, ++it) {
            const Tile ti = find_tile(gs, t);
            const int buf = it & 1;
            // the group's warps go on or leave together (this is also the tile's first barrier: the
            // staging buffer has been read)
            if (!group_all(h, warp_wait(&ctl.acc_full[buf], (it >> 1) & 1, abort))) {
                if (lane == 0) {
                    set_status(args.status, MOE_DEV_WAIT_TIMEOUT);
                    *abort = 1;
                }
                break;
            }
            tc_fence_after();
            const uint32_t acc = (buf ? kAccEnd - ti.nt : 0) + ((uint32_t)(q * 32) << 16);
            const int nch = ti.nt >> 5, h0 = h ^ (it & 1);  // chunks; the group's first one
            uint32_t r[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (h0 + 2 * i < nch) load_chunk<T>(acc + 32 * (h0 + 2 * i), r[i]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(&ctl.acc_empty[buf], 0);
            const int n0 = ti.n0 + (int)rank * 128;
            if (n0 < args.N) {
                T* out = static_cast<T*>(args.out) + (int64_t)ti.row0 * args.out_stride;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 32 * (h0 + 2 * i);
                    if (c < ti.nt)
                        store_chunk<T>(args, r[i], stage, out + c * args.out_stride, ti.rows - c, n0, q, h,
                                       lane, i == 0);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // Where a wait of this CTA ran out, copies that it issued after the leader had given up may be on
    // their way, counted on barriers of the leader's that nobody waits for: they land before it leaves
    // (a copy takes microseconds).
    if (*abort)
        for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < kCopyLandNs;) __nanosleep(1000);
    cluster_sync();  // the leader's MMAs have read this CTA's memory; both CTAs leave together
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(ctl.tmem, 512);
    }
}

// Two groups of four warps that wait as the epilogue does: warp 1's phase never completes, the
// others' has.  Bit w of *went_on: warp w passed its group's vote.
__global__ void __launch_bounds__(256) group_wait_probe_kernel(uint32_t* status, uint32_t* went_on,
                                                               uint64_t limit_ns)
{
    __shared__ uint64_t done, never;
    __shared__ int zero;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp >> 2;
    if (threadIdx.x == 0) {
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        zero = 0;
        fence_barrier_init();
        mbar_arrive(&done);
    }
    __syncthreads();
    const bool all = group_all(group, warp_wait(warp == 1 ? &never : &done, 0, &zero, limit_ns));
    if (lane == 0) {
        if (all) atomicOr(went_on, 1u << warp);
        else set_status(status, MOE_DEV_WAIT_TIMEOUT);
    }
}

MxGemmKernel gemm_mxfp4_kernel_for(int out_dtype)
{
    switch (out_dtype) {
        case MOE_BF16: return gemm_mxfp4_kernel<__nv_bfloat16>;
        case MOE_FP16: return gemm_mxfp4_kernel<__half>;
        default: return gemm_mxfp4_kernel<float>;
    }
}

}  // namespace moe
