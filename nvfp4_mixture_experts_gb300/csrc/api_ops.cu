// C ABI of the operators that need no handle: tokens sorted by expert and back with their
// gradients, MXFP4 and MXFP8 quantisation and the grouped products.  Argument checks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "host.cuh"

using namespace moe;

namespace {

int elem_bytes(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

bool dtype_ok(int dtype) { return dtype == MOE_BF16 || dtype == MOE_FP16 || dtype == MOE_FP32; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether an address is a multiple of an element's size (null: yes).
bool elem_aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// The same of arrays of 32-bit words: indices, counts, weights, status.
template <typename... P>
bool words_aligned(const P*... p)
{
    return (elem_aligned(p, 4) && ...);
}

// The largest power of two up to 16 that divides addresses, row sizes and strides (or-ed together).
int largest_unit(uint64_t ored) { return (int)((ored | 16) & (~(ored | 16) + 1)); }

uint64_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// Whether a tensor of rows can be moved in 16-byte pieces.
bool rows_vec(const void* p, int64_t row_bytes, int64_t stride_bytes)
{
    return aligned16(p) && row_bytes % 16 == 0 && stride_bytes % 16 == 0;
}

int num_sms()
{
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

unsigned blocks_for(int64_t work, int per_block, int per_sm)
{
    const int64_t want = (work + per_block - 1) / per_block;
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(want, (int64_t)num_sms() * per_sm));
}

// T, k, H and rows_cap of the sorted-row calls.
moe_status check_rows(int dtype, int T, int k, int H, int rows_cap)
{
    if (!dtype_ok(dtype) || T < 0 || k < 1 || H < 1 || rows_cap < 0) return MOE_ERR_INVALID;
    if (k > kMaxTopK || (int64_t)T * k > 0x7fffffff || H > (1 << 28)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Raises a kernel's limit of dynamic shared memory where the default (48 KB with the static part,
// up to 17 KB here) does not do.  The limit belongs to the kernel, not to a launch, so it is always
// raised to the `most` that any call takes: another thread's call between this and the launch may set
// it too, but not lower.
bool allow_smem(const void* kern, size_t bytes, size_t most)
{
    return bytes <= 31 * 1024 ||
           taken(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
}

// Blocks of the large sort's cluster: 16, more than the portable 8 (65536 pairs over 320 experts: 10.1
// us, 14.4 with 8; 16384: 6.5 and 7.6), where the device takes one such cluster with the most shared
// memory that a call wants (a part of a GPU may have no processing cluster of 16 SMs).  Asked once for a
// device; the debug flavour always takes 8, so that its tests run that form.  0: an error.
int sort_cluster_blocks(size_t most)
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (!taken(cudaGetDevice(&dev))) return 0;
    std::atomic<int>* slot = dev < 64 ? &known[dev] : nullptr;
    int blocks = slot ? slot->load(std::memory_order_relaxed) : 0;
    if (blocks) return blocks;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortBlocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortBlocks);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = most;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    // (a size that the device has no cluster of may be an error)
    const bool asked = taken(cudaOccupancyMaxActiveClusters(&clusters, sort_pairs_kernel, &cfg));
    blocks = asked && clusters > 0 && !kDebugChecks ? kSortBlocks : kSortBlocks / 2;
    if (slot) slot->store(blocks, std::memory_order_relaxed);
    return blocks;
}

bool align_ok(int a) { return a >= 1 && a <= 128 && (a & (a - 1)) == 0; }

// combine (w given) and dispatch's gradient (w null)
moe_status combine_rows(const void* y_d, int32_t dtype, const int32_t* inv_d, const float* w_d,
                        int32_t T, int32_t k, int32_t H, int32_t rows_cap, void* out_d,
                        int64_t out_stride, moe_stream_t stream)
{
    const moe_status st = check_rows(dtype, T, k, H, rows_cap);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    const int es = elem_bytes(dtype);
    if (!inv_d || !out_d || (rows_cap && !y_d) || (T > 1 && out_stride < H) ||
        !elem_aligned(y_d, es) || !elem_aligned(out_d, es) || !words_aligned(inv_d, w_d))
        return MOE_ERR_INVALID;
    const int unit = largest_unit(addr(y_d) | addr(out_d) | (uint64_t)H * es |
                                  (T > 1 ? (uint64_t)out_stride * es : 0));
    CombineArgs a = {};
    a.y = y_d;
    a.inv = inv_d;
    a.w = w_d;
    a.T = T;
    a.k = k;
    a.H = H;
    a.rows_cap = rows_cap;
    a.out = out_d;
    a.out_stride = out_stride;
    const int few = combine_few(k, T);
    const int64_t items = (int64_t)ceil_div(T, combine_tokens(few)) *
                          ceil_div((int)((int64_t)H * es / unit), combine_run(unit));
    return launch(combine_rows_kernel_for(dtype, unit, few), dim3(blocks_for(items, 8, 16)), dim3(256), 0,
                  reinterpret_cast<cudaStream_t>(stream), true, a);
}

// moe_quant_mxfp4, and (eight_bits) moe_quant_mxfp8
moe_status quant_rows(bool eight_bits, const void* x_d, int32_t dtype, int32_t batch, int32_t rows,
                      int32_t cols, int64_t row_stride, int64_t batch_stride, int32_t transpose,
                      int32_t scale_rule, const int32_t* perm_src_d, uint8_t* codes_d, uint8_t* sf_d,
                      int32_t sf_layout, void* values_d, moe_stream_t stream)
{
    if (!dtype_ok(dtype) || batch < 0 || rows < 0 || cols < 1) return MOE_ERR_INVALID;
    if (transpose != 0 && transpose != 1) return MOE_ERR_INVALID;
    if (scale_rule != MOE_MX_FLOOR && scale_rule != MOE_MX_CEIL) return MOE_ERR_INVALID;
    if (sf_layout != MOE_SF_CANONICAL && sf_layout != MOE_SF_TILED) return MOE_ERR_INVALID;
    if (perm_src_d && (transpose || batch != 1)) return MOE_ERR_INVALID;
    if ((transpose ? rows : cols) % 32) return MOE_ERR_UNSUPPORTED;
    if (batch == 0 || rows == 0) return MOE_OK;
    if (!x_d || !codes_d || !sf_d || (rows > 1 && row_stride < cols) ||
        (batch > 1 && batch_stride < 0))
        return MOE_ERR_INVALID;
    if (!aligned16(codes_d) || (values_d && !aligned16(values_d)) ||
        (sf_layout == MOE_SF_TILED && !aligned16(sf_d)) || !elem_aligned(x_d, elem_bytes(dtype)) ||
        !words_aligned(perm_src_d))
        return MOE_ERR_INVALID;
    MxQuantArgs a = {};
    a.x = x_d;
    a.row_stride = row_stride;
    a.batch_stride = batch_stride;
    a.batch = batch;
    a.rows = rows;
    a.cols = cols;
    a.rule = scale_rule;
    a.perm_src = perm_src_d;
    a.codes = codes_d;
    a.sf = sf_d;
    a.layout = sf_layout;
    a.values = values_d;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int es = elem_bytes(dtype);
    if (transpose) {
        const int64_t tiles = (int64_t)batch * ceil_div(rows, 128) * ceil_div(cols, mx_transposed_cols(es));
        // 16-bit types: two neighbouring columns are one aligned word in every row
        const bool words = addr(x_d) % 4 == 0 && row_stride % 2 == 0 && (batch == 1 || batch_stride % 2 == 0);
        const MxQuantKernel kern = mx_quant_transposed_kernel_for(dtype, words);
        const size_t smem = mx_transposed_smem(es);
        if (!allow_smem(reinterpret_cast<const void*>(kern), smem, smem)) return MOE_ERR_CUDA;
        return launch(kern, dim3(blocks_for(tiles, 1, 16)), dim3(256), smem, s, true, a);
    }
    const bool vec = rows_vec(x_d, (int64_t)cols * es, rows > 1 ? row_stride * es : 0) &&
                     (batch == 1 || batch_stride * es % 16 == 0);
    // The kernel for long rows keeps a warp's runs in one row: it wants rows that fill half of their
    // runs or more (bf16 with values, this and the other: 5000 x 3584 14.4 and 17.1 us, 16384 x 512
    // 8.6 and 8.7, 30000 x 256 9.7 and 8.2, 262144 x 32 63 and 9.7) and enough of them to fill the GPU
    // (8192 x 4096 24.4 and 30.3, 2048 x 2048 4.7 and 4.9, 64 x 4096 2.3 and 1.6).
    if ((int64_t)batch * rows > 0xffffffffll) return MOE_ERR_UNSUPPORTED;
    const int64_t eights = (int64_t)batch * rows * (cols / 8);
    const int runs = ceil_div(cols / 8, kMxQuantRun);
    const bool short_rows =
        eights < (1 << 19) ||
        (eights <= 0xffffffffll && 2 * (cols / 8) < runs * (int64_t)kMxQuantRun);
    const int64_t items = short_rows ? eights : (int64_t)batch * rows * runs;
    if (items > 0xffffffffll) return MOE_ERR_UNSUPPORTED;
    return launch(mx_quant_kernel_for(eight_bits, dtype, vec, short_rows),
                  dim3(blocks_for(items, short_rows ? 256 : 8, 16)), dim3(256), 0, s, true, a);
}

// moe_grouped_gemm_mxfp4, and (eight_bits) moe_grouped_gemm_mxfp8
moe_status grouped_gemm(bool eight_bits, const uint8_t* a_codes_d, const uint8_t* a_sf_d, int32_t rows_cap,
                        const int32_t* counts_d, const int32_t* offsets_d, int32_t num_groups,
                        const uint8_t* w_codes_d, const uint8_t* w_sf_d, int32_t N, int32_t K, void* out_d,
                        int32_t out_dtype, int64_t out_stride, void* ws_d, size_t ws_bytes,
                        uint32_t* status_d, moe_stream_t stream)
{
    if (!dtype_ok(out_dtype) || rows_cap < 0 || num_groups < 1 || N < 1 || K < 1 ||
        !counts_d != !offsets_d || (!counts_d && num_groups != 1))
        return MOE_ERR_INVALID;
    if (K % (eight_bits ? 128 : 32) || num_groups > kMaxExperts || (int64_t)num_groups * N > 0x7fffffff)
        return MOE_ERR_UNSUPPORTED;
    if (rows_cap == 0) return MOE_OK;
    if (!a_codes_d || !a_sf_d || !w_codes_d || !w_sf_d || !out_d ||
        (rows_cap > 1 && out_stride < N))
        return MOE_ERR_INVALID;
    if (!aligned16(a_codes_d) || !aligned16(a_sf_d) || !aligned16(w_codes_d) || !aligned16(w_sf_d) ||
        (eight_bits && addr(w_codes_d) % 32) ||
        (reinterpret_cast<uintptr_t>(out_d) % elem_bytes(out_dtype)) != 0 ||
        (reinterpret_cast<uintptr_t>(ws_d) & 255) != 0 || (ws_bytes && !ws_d) ||
        !words_aligned(counts_d, offsets_d, status_d))
        return MOE_ERR_INVALID;
    const int KA = (K / 32 + 3) / 4, es = elem_bytes(out_dtype);
    CUtensorMap tmW, tmT, tmT16, tmT32, tmT64, tmSW, tmST;
    constexpr auto U32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
    constexpr auto SW = CU_TENSOR_MAP_SWIZZLE_128B, NOSW = CU_TENSOR_MAP_SWIZZLE_NONE;
    // 16U4_ALIGN16B: 16 packed codes become 16 bytes of shared memory (8 of them padding), as
    // kind::mxf8f6f4 reads E2M1 operands
    constexpr auto U4 = CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B;
    const uint64_t row = eight_bits ? K : K / 2;   // bytes of a group row
    if (!(eight_bits ? make_tmap_3d(&tmW, w_codes_d, U4, K, N, num_groups, K / 2, 128, 128, SW)
                     : make_tmap_3d(&tmW, w_codes_d, U32, K / 8, N, num_groups, K / 2, 32, 128, SW)) ||
        !make_tmap(&tmT, a_codes_d, U32, row / 4, rows_cap, row, 32, 128, SW) ||
        !make_tmap(&tmT16, a_codes_d, U32, row / 4, rows_cap, row, 32, 16, SW) ||
        (eight_bits && (!make_tmap(&tmT32, a_codes_d, U32, row / 4, rows_cap, row, 32, 32, SW) ||
                        !make_tmap(&tmT64, a_codes_d, U32, row / 4, rows_cap, row, 32, 64, SW))) ||
        !make_tmap(&tmSW, w_sf_d, U32, KA * 128, (uint64_t)num_groups * ceil_div(N, 128), (uint64_t)KA * 512,
                   256, 1, NOSW) ||
        !make_tmap(&tmST, a_sf_d, U32, KA * 128, ceil_div(rows_cap, 128), (uint64_t)KA * 512, 256, 1, NOSW))
        return MOE_ERR_CUDA;
    if (!eight_bits) tmT32 = tmT64 = tmT16;  // (not used)
    MxGemmArgs a = {};
    a.rows_cap = rows_cap;
    a.counts = counts_d;
    a.offsets = offsets_d;
    a.G = num_groups;
    a.N = N;
    a.K = K;
    a.out = out_d;
    a.out_stride = out_stride;
    a.unit = largest_unit(addr(out_d) | (uint64_t)N * es | (rows_cap > 1 ? (uint64_t)out_stride * es : 0));
    if (a.unit == 8) a.unit = 4;
    a.status = status_d;
    const MxGemmKernel kern = gemm_mxfp4_kernel_for(eight_bits, out_dtype);
    a.stages = kMxStages;
    while (gemm_mxfp4_smem(a.stages, num_groups, es) > kSmemLimit) --a.stages;  // over 618 groups: 5
    const int smem = gemm_mxfp4_smem(a.stages, num_groups, es);
    if (!allow_smem(reinterpret_cast<const void*>(kern), smem, kSmemLimit)) return MOE_ERR_CUDA;
    // at most this many tiles, however the rows fall into groups
    const int64_t tiles = std::min<int64_t>(num_groups + rows_cap / kMxTileRows, ceil_div(rows_cap, 128)) *
                          ceil_div(N, 256);
    const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, num_sms() / 2));
    return launch_pairs(kern, dim3(2 * pairs), dim3(kMxThreads), smem,
                        reinterpret_cast<cudaStream_t>(stream), true, tmW, tmT, tmT16, tmT32, tmT64, tmSW, tmST,
                        a);
}

// What the calls with an MX result share: its layout and rule, and the addresses of an MXFP8 matrix
// (null: none).
bool mx_choice_ok(int sf_layout, int scale_rule)
{
    return (scale_rule == MOE_MX_FLOOR || scale_rule == MOE_MX_CEIL) &&
           (sf_layout == MOE_SF_CANONICAL || sf_layout == MOE_SF_TILED);
}

bool mx8_aligned(const uint8_t* codes, const uint8_t* sf, int sf_layout)
{
    return aligned16(codes) && (sf_layout != MOE_SF_TILED || aligned16(sf));
}

moe_status check_route(int dtype, int T, int E, int k, int score, int renorm)
{
    if (!dtype_ok(dtype) || T < 0 || E < 1 || k < 1 || k > E ||
        (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || (renorm != 0 && renorm != 1))
        return MOE_ERR_INVALID;
    return E > kMaxExperts || k > kMaxTopK ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_norm(int dtype, int T, int H)
{
    if (!dtype_ok(dtype) || T < 0 || H < 1) return MOE_ERR_INVALID;
    return H > kNormMost ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_swiglu(int dtype, int rows, int inter, int sf_layout, int scale_rule)
{
    if (!dtype_ok(dtype) || rows < 0 || inter < 1 || !mx_choice_ok(sf_layout, scale_rule)) return MOE_ERR_INVALID;
    return inter % 32 || inter > (1 << 28) || (int64_t)rows * (inter / 8) > 0xffffffffll ? MOE_ERR_UNSUPPORTED
                                                                                         : MOE_OK;
}

}  // namespace

extern "C" {

int32_t moe_dispatch_rows_capacity(int32_t T, int32_t k, int32_t num_local, int32_t row_align)
{
    if (T < 0 || k < 1 || k > kMaxTopK || num_local < 0 || num_local > kMaxExperts ||
        !align_ok(row_align))
        return 0;
    const int64_t P = (int64_t)T * k, a = row_align;
    const int64_t rows = (P + std::min<int64_t>(num_local, P) * (a - 1) + a - 1) / a * a;
    return rows > 0x7fffffff ? 0 : (int32_t)rows;
}

moe_status moe_dispatch(const void* x_d, int32_t dtype, int64_t x_stride,
                        const int32_t* topk_ids_d, int32_t T, int32_t k, int32_t H,
                        int32_t num_experts, int32_t local_off, int32_t num_local,
                        int32_t row_align, int32_t rows_cap, int32_t* counts_d,
                        int32_t* offsets_d, int32_t* perm_src_d, int32_t* inv_d, void* rows_d,
                        uint32_t* status_d, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_dispatch");
    const bool move = x_d && rows_d;  // (a tensor of no tokens or of no rows may have no address)
    if (!move && ((rows_d && T > 0) || (x_d && rows_cap > 0))) return MOE_ERR_INVALID;
    const moe_status st = check_rows(move ? dtype : MOE_BF16, T, k, move ? H : 1, rows_cap);
    if (st != MOE_OK) return st;
    if (num_experts < 1 || local_off < 0 || num_local < 0 || !align_ok(row_align) ||
        (int64_t)local_off + num_local > num_experts || k > num_experts)
        return MOE_ERR_INVALID;
    if (move && T > 1 && x_stride < H) return MOE_ERR_INVALID;
    if (!offsets_d || (num_local && !counts_d) || (T && (!topk_ids_d || !inv_d)) ||
        (rows_cap && !perm_src_d) ||
        !words_aligned(topk_ids_d, counts_d, offsets_d, perm_src_d, inv_d, status_d))
        return MOE_ERR_INVALID;
    if (move && (!elem_aligned(x_d, elem_bytes(dtype)) || !elem_aligned(rows_d, elem_bytes(dtype))))
        return MOE_ERR_INVALID;
    const int64_t P = (int64_t)T * k;
    if (num_experts > kMaxExperts || P + (int64_t)num_local * (row_align - 1) > 0x7fffffff)
        return MOE_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    SortArgs a = {};
    a.ids = topk_ids_d;
    a.P = (int)P;
    a.E = num_experts;
    a.off = local_off;
    a.El = num_local;
    a.align = row_align;
    a.rows_cap = rows_cap;
    a.counts = counts_d;
    a.offsets = offsets_d;
    a.perm_src = perm_src_d;
    a.inv = inv_d;
    a.status = status_d;
    DispatchArgs d = {};
    int unit = 16;
    if (move) {
        const int es = elem_bytes(dtype);
        unit = largest_unit(addr(x_d) | addr(rows_d) | (uint64_t)H * es | (T > 1 ? (uint64_t)x_stride * es : 0));
        d.x = x_d;
        d.x_stride = x_stride * es / unit;
        d.inv = inv_d;
        d.T = T;
        d.k = k;
        d.units = (int)((int64_t)H * es / unit);
        d.rows_cap = rows_cap;
        d.perm_src = perm_src_d;
        d.rows = rows_d;
    }
    const bool small = P <= kSmallPairs;
    const size_t smem = sort_smem(num_local, small ? ceil_div((int)P, 32) : 32);
    const size_t most = sort_smem(kMaxExperts, 32);
    if (small) {
        a.segment = 32;
        const DispatchSmallKernel kern = dispatch_small_kernel_for(unit);
        if (!allow_smem(reinterpret_cast<const void*>(kern), smem, most)) return MOE_ERR_CUDA;
        const int blocks = std::max(1, std::min(move ? T : ceil_div(rows_cap, 8192), num_sms()));
        return launch(kern, dim3(blocks), dim3(kSortThreads), smem, s, true, a, d);
    }
    a.rows_follow = move && rows_cap > 0 && num_local > 0;
    if (!allow_smem(reinterpret_cast<const void*>(sort_pairs_kernel), most, most) ||
        !taken(cudaFuncSetAttribute(sort_pairs_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)))
        return MOE_ERR_CUDA;
    const int blocks = sort_cluster_blocks(most);
    if (!blocks) return MOE_ERR_CUDA;
    a.segment = ceil_div((int)((P + 31) / 32), blocks * 32) * 32;
    const moe_status sorted = launch_cluster(sort_pairs_kernel, blocks, dim3(blocks),
                                             dim3(kSortThreads), smem, s, true, a);
    if (sorted != MOE_OK || !a.rows_follow) return sorted;
    const int64_t runs = (int64_t)T * ceil_div(d.units, kDispatchRun);
    return launch(dispatch_rows_kernel_for(unit), dim3(blocks_for(runs, 8, 16)), dim3(256), 0, s,
                  true, d);
}

moe_status moe_dispatch_backward(const void* drows_d, int32_t dtype, const int32_t* inv_d,
                                 int32_t T, int32_t k, int32_t H, int32_t rows_cap, void* dx_d,
                                 int64_t dx_stride, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_dispatch_backward");
    return combine_rows(drows_d, dtype, inv_d, nullptr, T, k, H, rows_cap, dx_d, dx_stride, stream);
}

moe_status moe_combine_weighted(const void* y_d, int32_t dtype, const int32_t* inv_d,
                                const float* w_d, int32_t T, int32_t k, int32_t H,
                                int32_t rows_cap, void* out_d, int64_t out_stride,
                                moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_combine_weighted");
    if (T > 0 && !w_d) return MOE_ERR_INVALID;
    return combine_rows(y_d, dtype, inv_d, w_d, T, k, H, rows_cap, out_d, out_stride, stream);
}

moe_status moe_combine_backward(const void* dout_d, int32_t dtype, int64_t dout_stride,
                                const void* y_d, const int32_t* inv_d, const float* w_d,
                                int32_t T, int32_t k, int32_t H, int32_t rows_cap, void* dy_d,
                                float* dw_d, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_combine_backward");
    const moe_status st = check_rows(dtype, T, k, H, rows_cap);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!dy_d && !dw_d && rows_cap == 0) return MOE_OK;  // (dy has no rows, so it may have no address)
    if (!dout_d || !inv_d || !w_d || (!dy_d && !dw_d) || (dw_d && rows_cap && !y_d) ||
        (T > 1 && dout_stride < H))
        return MOE_ERR_INVALID;
    const int es = elem_bytes(dtype);
    if (!elem_aligned(dout_d, es) || !elem_aligned(y_d, es) || !elem_aligned(dy_d, es) ||
        !words_aligned(inv_d, w_d, dw_d))
        return MOE_ERR_INVALID;
    const int unit = largest_unit(addr(dout_d) | (dw_d ? addr(y_d) : 0) | addr(dy_d) | (uint64_t)H * es |
                                  (T > 1 ? (uint64_t)dout_stride * es : 0));
    CombineBackArgs a = {};
    a.dout = dout_d;
    a.dout_stride = dout_stride;
    a.y = y_d;
    a.inv = inv_d;
    a.w = w_d;
    a.T = T;
    a.k = k;
    a.H = H;
    a.rows_cap = rows_cap;
    a.dy = dy_d;
    a.dw = dw_d;
    // Rows of over 4.5 KB and more than four pairs a token: the kernel that takes all pairs at once
    // (k 8, bf16, 8192 tokens x 4096: 170 us, 182 with the one that takes the kept pairs four at a
    // time; x 3000: 132 and 140).  Else the latter (x 2056, 3 of 8 pairs kept: 46 us, 53 with the
    // former; x 304, k 6, 2 of 6 kept: 8.6 and 15).
    const int64_t row = (int64_t)H * es;
    const bool all = k > 4 && row > 4608;
    // Warps per token (or batch of tokens): one, for long rows two, or as many more as give every SM
    // its 16: a token's warps wait for one another at its end (7003 tokens x 1096, k 3: one warp 20.7
    // us, two 24.5; 8192 x 4001, k 8: 275 and 258), but few tokens' latency counts (64 tokens x 4096,
    // k 8: two warps 6.7 us, eight 3.8).
    const int few = combine_few(k, T), batches = ceil_div(T, combine_tokens(few));
    int warps = row <= 6144 && !all ? 1 : 2;
    while (warps < 8 && (int64_t)batches * warps < 16 * num_sms()) warps *= 2;
    return launch(combine_back_kernel_for(dtype, unit, warps, few, all),
                  dim3(blocks_for(batches, 1, 64 / warps)), dim3(32 * warps), 0,
                  reinterpret_cast<cudaStream_t>(stream), true, a);
}

size_t moe_mxfp4_scale_bytes(int32_t batch, int32_t rows, int32_t cols, int32_t sf_layout)
{
    if (batch < 0 || rows < 0 || cols <= 0 || cols % 32 ||
        (sf_layout != MOE_SF_CANONICAL && sf_layout != MOE_SF_TILED))
        return 0;
    const size_t blocks = (size_t)cols / 32;
    if (sf_layout == MOE_SF_CANONICAL) return (size_t)batch * rows * blocks;
    return (size_t)batch * (((size_t)rows + 127) / 128) * ((blocks + 3) / 4) * 512;
}

moe_status moe_quant_mxfp4(const void* x_d, int32_t dtype, int32_t batch, int32_t rows,
                           int32_t cols, int64_t row_stride, int64_t batch_stride,
                           int32_t transpose, int32_t scale_rule, const int32_t* perm_src_d,
                           uint8_t* codes_d, uint8_t* sf_d, int32_t sf_layout, void* values_d,
                           moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_quant_mxfp4");
    return quant_rows(false, x_d, dtype, batch, rows, cols, row_stride, batch_stride, transpose, scale_rule,
                      perm_src_d, codes_d, sf_d, sf_layout, values_d, stream);
}

moe_status moe_quant_mxfp8(const void* x_d, int32_t dtype, int32_t batch, int32_t rows,
                           int32_t cols, int64_t row_stride, int64_t batch_stride,
                           int32_t scale_rule, const int32_t* perm_src_d, uint8_t* codes_d,
                           uint8_t* sf_d, int32_t sf_layout, void* values_d, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_quant_mxfp8");
    return quant_rows(true, x_d, dtype, batch, rows, cols, row_stride, batch_stride, 0, scale_rule,
                      perm_src_d, codes_d, sf_d, sf_layout, values_d, stream);
}

moe_status moe_mxfp4_tile_scales(const uint8_t* sf_d, int32_t batch, int32_t rows, int32_t cols,
                                 uint8_t* sf_tiled_d, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_mxfp4_tile_scales");
    if (batch < 0 || rows < 0 || cols < 1) return MOE_ERR_INVALID;
    if (cols % 32) return MOE_ERR_UNSUPPORTED;
    if (batch == 0 || rows == 0) return MOE_OK;
    if (!sf_d || !sf_tiled_d || !aligned16(sf_tiled_d)) return MOE_ERR_INVALID;
    const int64_t n = (int64_t)moe_mxfp4_scale_bytes(batch, rows, cols, MOE_SF_TILED) / 4;
    return launch(mx_tile_scales_kernel, dim3(blocks_for(n, 256, 16)), dim3(256), 0,
                  reinterpret_cast<cudaStream_t>(stream), false, sf_d, batch, rows, cols / 32,
                  sf_tiled_d);
}

size_t moe_mxfp4_workspace_size(int32_t rows_cap, int32_t num_groups, int32_t N, int32_t K)
{
    (void)rows_cap, (void)num_groups, (void)N, (void)K;
    return 0;
}

moe_status moe_grouped_gemm_mxfp4(const uint8_t* a_codes_d, const uint8_t* a_sf_d,
                                  int32_t rows_cap, const int32_t* counts_d,
                                  const int32_t* offsets_d, int32_t num_groups,
                                  const uint8_t* w_codes_d, const uint8_t* w_sf_d, int32_t N,
                                  int32_t K, void* out_d, int32_t out_dtype, int64_t out_stride,
                                  void* ws_d, size_t ws_bytes, uint32_t* status_d,
                                  moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_grouped_gemm_mxfp4");
    return grouped_gemm(false, a_codes_d, a_sf_d, rows_cap, counts_d, offsets_d, num_groups, w_codes_d, w_sf_d,
                        N, K, out_d, out_dtype, out_stride, ws_d, ws_bytes, status_d, stream);
}

moe_status moe_grouped_gemm_mxfp8(const uint8_t* a_codes_d, const uint8_t* a_sf_d,
                                  int32_t rows_cap, const int32_t* counts_d,
                                  const int32_t* offsets_d, int32_t num_groups,
                                  const uint8_t* w_codes_d, const uint8_t* w_sf_d, int32_t N,
                                  int32_t K, void* out_d, int32_t out_dtype, int64_t out_stride,
                                  uint32_t* status_d, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_grouped_gemm_mxfp8");
    return grouped_gemm(true, a_codes_d, a_sf_d, rows_cap, counts_d, offsets_d, num_groups, w_codes_d, w_sf_d,
                        N, K, out_d, out_dtype, out_stride, nullptr, 0, status_d, stream);
}

moe_status moe_route_scores(const void* logits_d, int32_t dtype, int64_t stride, const float* bias_d,
                            int32_t T, int32_t num_experts, int32_t k, int32_t score,
                            int32_t num_groups, int32_t topk_groups, int32_t group_score,
                            int32_t renormalise, float scale, int32_t* topk_ids_d, float* topk_w_d,
                            moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_route_scores");
    const moe_status st = check_route(dtype, T, num_experts, k, score, renormalise);
    if (st != MOE_OK) return st;
    if (num_groups < 1 || num_experts % num_groups || topk_groups < 1 || topk_groups > num_groups ||
        (int64_t)topk_groups * (num_experts / num_groups) < k ||
        (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2))
        return MOE_ERR_INVALID;
    if (num_groups > kRouteGroups) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!logits_d || !topk_ids_d || !topk_w_d || (T > 1 && stride < num_experts) ||
        !elem_aligned(logits_d, elem_bytes(dtype)) || !words_aligned(bias_d, topk_ids_d, topk_w_d))
        return MOE_ERR_INVALID;
    RouteArgs a = {};
    a.logits = logits_d;
    a.stride = stride;
    a.bias = bias_d;
    a.T = T;
    a.E = num_experts;
    a.k = k;
    a.score = score;
    a.groups = topk_groups == num_groups ? 1 : num_groups;  // (of all groups: no choice among them)
    a.topk_groups = a.groups == 1 ? 1 : topk_groups;
    a.group_score = group_score;
    a.group = num_experts / num_groups;
    a.group_mul = ((1u << 20) + a.group - 1) / a.group;
    a.renorm = renormalise;
    a.scale = scale;
    a.ids = topk_ids_d;
    a.w = topk_w_d;
    const RouteKernel kern = route_scores_kernel_for(dtype, num_experts);
    const size_t smem = route_smem(num_experts, a.groups);
    if (!allow_smem(reinterpret_cast<const void*>(kern), smem, route_smem(kMaxExperts, 2))) return MOE_ERR_CUDA;
    return launch(kern, dim3(ceil_div(T, kRouteWarps)), dim3(32 * kRouteWarps), smem,
                  reinterpret_cast<cudaStream_t>(stream), true, a);
}

moe_status moe_route_scores_backward(const void* logits_d, int32_t dtype, int64_t stride,
                                     const int32_t* topk_ids_d, const float* dtopk_w_d, int32_t T,
                                     int32_t num_experts, int32_t k, int32_t score,
                                     int32_t renormalise, float scale, void* dlogits_d,
                                     int64_t dstride, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_route_scores_backward");
    const moe_status st = check_route(dtype, T, num_experts, k, score, renormalise);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    const int es = elem_bytes(dtype);
    if (!logits_d || !topk_ids_d || !dtopk_w_d || !dlogits_d ||
        (T > 1 && (stride < num_experts || dstride < num_experts)) || !elem_aligned(logits_d, es) ||
        !elem_aligned(dlogits_d, es) || !words_aligned(topk_ids_d, dtopk_w_d))
        return MOE_ERR_INVALID;
    RouteBackArgs a = {};
    a.logits = logits_d;
    a.stride = stride;
    a.ids = topk_ids_d;
    a.dw = dtopk_w_d;
    a.T = T;
    a.E = num_experts;
    a.k = k;
    a.score = score;
    a.renorm = renormalise;
    a.scale = scale;
    a.dlogits = dlogits_d;
    a.dstride = dstride;
    return launch(route_back_kernel_for(dtype, score == MOE_SCORE_SOFTMAX && !renormalise, num_experts), dim3(ceil_div(T, kRouteWarps)), dim3(32 * kRouteWarps), 0,
                  reinterpret_cast<cudaStream_t>(stream), true, a);
}

moe_status moe_rmsnorm(const void* x_d, int32_t dtype, int64_t x_stride, const void* residual_d,
                       int64_t residual_stride, const void* weight_d, float eps, int32_t T, int32_t H,
                       void* h_d, int64_t h_stride, void* y_d, int64_t y_stride, float* rstd_d,
                       uint8_t* codes_d, uint8_t* sf_d, int32_t sf_layout, int32_t scale_rule,
                       moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_rmsnorm");
    const moe_status st = check_norm(dtype, T, H);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.0f) || (h_d && !residual_d) || !codes_d != !sf_d || !mx_choice_ok(sf_layout, scale_rule) ||
        (!y_d && !codes_d && !h_d && !rstd_d && T > 0))
        return MOE_ERR_INVALID;
    if (codes_d && H % 32) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    const int es = elem_bytes(dtype);
    if (!x_d || (T > 1 && (x_stride < H || (residual_d && residual_stride < H) || (h_d && h_stride < H) ||
                           (y_d && y_stride < H))) ||
        !elem_aligned(x_d, es) || !elem_aligned(residual_d, es) || !elem_aligned(weight_d, es) ||
        !elem_aligned(h_d, es) || !elem_aligned(y_d, es) || !words_aligned(rstd_d) ||
        !mx8_aligned(codes_d, sf_d, sf_layout))
        return MOE_ERR_INVALID;
    NormArgs a = {};
    a.x = x_d;
    a.x_stride = x_stride;
    a.res = residual_d;
    a.res_stride = residual_stride;
    a.w = weight_d;
    a.eps = eps;
    a.T = T;
    a.H = H;
    a.h = h_d;
    a.h_stride = h_stride;
    a.y = y_d;
    a.y_stride = y_stride;
    a.rstd = rstd_d;
    a.codes = codes_d;
    a.sf = sf_d;
    a.layout = sf_layout;
    a.rule = scale_rule;
    const uint64_t some = T > 1 ? es : 0;   // (of one row strides are of no effect)
    int piece = largest_unit(addr(x_d) | addr(residual_d) | addr(weight_d) | addr(h_d) | addr(y_d) |
                                   (uint64_t)H * es | x_stride * some | (residual_d ? residual_stride * some : 0) |
                                   (h_d ? h_stride * some : 0) | (y_d ? y_stride * some : 0));
    if (H <= kNormShort && H % 8) piece = std::min(piece, 8);  // (a warp's eights are whole)
    const int threads = norm_threads(H);
    // (fp32 rows of an odd number of 16-byte pieces have no whole eights: in the ring, whatever it takes)
    if (piece == 16 && H > kNormShort) {
        a.depth = norm_depth(threads, es, residual_d ? 2 : 1);
        if (!a.depth && H % 8) a.depth = 1;
    }
    const NormKernel kern = norm_kernel_for(dtype, H, piece, codes_d != nullptr, threads, a.depth > 0);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!a.depth)
        return launch(kern, dim3(H <= kNormShort ? ceil_div(T, 8) : T), dim3(threads), 0, s, true, a);
    const size_t smem = (size_t)a.depth * norm_row_bytes(threads, es, 2);  // (room for both, whatever is given)
    if (!allow_smem(reinterpret_cast<const void*>(kern), smem, kNormRingMost)) return MOE_ERR_CUDA;
    return launch(kern, dim3(std::min(T, num_sms() * norm_per_sm(threads, false))), dim3(threads), smem, s, true, a);
}

size_t moe_rmsnorm_workspace_size(int32_t T, int32_t H)
{
    if (check_norm(MOE_BF16, T, H) != MOE_OK) return 0;
    const int parts = norm_parts(T, H, H <= kNormShort);  // (no fewer than of warps, where those have longer rows)
    return parts > 1 ? (size_t)parts * H * 4 : 0;
}

moe_status moe_rmsnorm_backward(const void* dy_d, int32_t dtype, int64_t dy_stride, const void* dh_d,
                                int64_t dh_stride, const void* h_d, int64_t h_stride,
                                const void* weight_d, const float* rstd_d, int32_t T, int32_t H,
                                void* dx_d, int64_t dx_stride, float* dweight_d, void* ws_d,
                                size_t ws_bytes, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_rmsnorm_backward");
    const moe_status st = check_norm(dtype, T, H);
    if (st != MOE_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!words_aligned(dweight_d, rstd_d)) return MOE_ERR_INVALID;
    if (T == 0) {
        if (!dweight_d) return MOE_OK;
        return taken(cudaMemsetAsync(dweight_d, 0, (size_t)H * 4, s)) ? MOE_OK : MOE_ERR_CUDA;
    }
    const int es = elem_bytes(dtype);
    if (!dy_d || !h_d || !rstd_d || !dx_d ||
        (T > 1 && (dy_stride < H || h_stride < H || dx_stride < H || (dh_d && dh_stride < H))) ||
        !elem_aligned(dy_d, es) || !elem_aligned(dh_d, es) || !elem_aligned(h_d, es) ||
        !elem_aligned(weight_d, es) || !elem_aligned(dx_d, es) || (ws_bytes && !ws_d) || (addr(ws_d) & 255))
        return MOE_ERR_INVALID;
    if (dweight_d && ws_bytes < moe_rmsnorm_workspace_size(T, H)) return MOE_ERR_WORKSPACE;
    NormBackArgs a = {};
    a.dy = dy_d;
    a.dy_stride = dy_stride;
    a.h = h_d;
    a.h_stride = h_stride;
    a.w = weight_d;
    a.rstd = rstd_d;
    a.dh = dh_d;
    a.dh_stride = dh_stride;
    a.T = T;
    a.H = H;
    a.dx = dx_d;
    a.dx_stride = dx_stride;
    a.dw = dweight_d;
    a.ws = static_cast<float*>(ws_d);
    const uint64_t some = T > 1 ? es : 0;
    const int piece = largest_unit(addr(dy_d) | addr(dh_d) | addr(h_d) | addr(weight_d) | addr(dx_d) |
                                   (uint64_t)H * es | dy_stride * some | h_stride * some | dx_stride * some |
                                   (dh_d ? dh_stride * some : 0));
    const int threads = norm_threads(H);
    const bool one = norm_back_one(H, piece, es);
    const NormBackKernel kern = norm_back_kernel_for(dtype, H, piece, threads);
    a.parts = norm_parts(T, H, one);
    size_t smem = 0;
    if (piece == 16) {
        a.depth = norm_back_depth(H, es, one);
        smem = (size_t)a.depth * norm_back_row_bytes(H, es, one);
        if (!allow_smem(reinterpret_cast<const void*>(kern), smem, kNormRingMost)) return MOE_ERR_CUDA;
    }
    const moe_status done = launch(kern, dim3(a.parts), dim3(one ? 256 : threads), smem, s, true, a);
    if (done != MOE_OK || !dweight_d || a.parts == 1) return done;
    return launch(norm_parts_kernel, dim3(ceil_div(H, 8)), dim3(256), 0, s, true, a.ws, a.parts, H, dweight_d);
}

moe_status moe_swiglu_mxfp8(const void* gate_up_d, int32_t dtype, int64_t stride, int32_t rows, int32_t inter,
                            const int32_t* perm_src_d, int32_t scale_rule, uint8_t* codes_d, uint8_t* sf_d,
                            int32_t sf_layout, uint8_t* ckpt_d, uint8_t* ckpt_sf_d, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_swiglu_mxfp8");
    const moe_status st = check_swiglu(dtype, rows, inter, sf_layout, scale_rule);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (!gate_up_d || !codes_d || !sf_d || !ckpt_d != !ckpt_sf_d || (rows > 1 && stride < 2 * (int64_t)inter) ||
        !elem_aligned(gate_up_d, elem_bytes(dtype)) || !words_aligned(perm_src_d) ||
        !mx8_aligned(codes_d, sf_d, sf_layout) || !mx8_aligned(ckpt_d, ckpt_sf_d, MOE_SF_CANONICAL))
        return MOE_ERR_INVALID;
    SwigluArgs a = {};
    a.gu = gate_up_d;
    a.gu_stride = stride;
    a.rows = rows;
    a.inter = inter;
    a.n = (uint32_t)((int64_t)rows * (inter / 16));
    a.units = FastDiv(inter / 16);
    a.rule = scale_rule;
    a.perm_src = perm_src_d;
    a.codes = codes_d;
    a.sf = sf_d;
    a.layout = sf_layout;
    a.ckpt = ckpt_d;
    a.ckpt_sf = ckpt_sf_d;
    const int es = elem_bytes(dtype);
    const bool vec = rows_vec(gate_up_d, (int64_t)inter * es, rows > 1 ? stride * es : 0);
    return launch(swiglu_kernel_for(dtype, vec), dim3(blocks_for((int64_t)rows * (inter / 16), 256, 8)),
                  dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), true, a);
}

moe_status moe_swiglu_mxfp8_backward(const void* ds_d, int32_t dtype, int64_t stride, const uint8_t* ckpt_d,
                                     const uint8_t* ckpt_sf_d, int32_t rows, int32_t inter,
                                     const int32_t* perm_src_d, int32_t scale_rule, uint8_t* codes_d,
                                     uint8_t* sf_d, int32_t sf_layout, void* dgate_up_d, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_swiglu_mxfp8_backward");
    const moe_status st = check_swiglu(dtype, rows, inter, sf_layout, scale_rule);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (!ds_d || !ckpt_d || !ckpt_sf_d || !codes_d != !sf_d || (!codes_d && !dgate_up_d) ||
        (rows > 1 && stride < inter) || !elem_aligned(ds_d, elem_bytes(dtype)) || !words_aligned(perm_src_d) ||
        !mx8_aligned(codes_d, sf_d, sf_layout) || !mx8_aligned(ckpt_d, ckpt_sf_d, MOE_SF_CANONICAL) ||
        !aligned16(dgate_up_d))
        return MOE_ERR_INVALID;
    SwigluBackArgs a = {};
    a.ds = ds_d;
    a.ds_stride = stride;
    a.ckpt = ckpt_d;
    a.ckpt_sf = ckpt_sf_d;
    a.rows = rows;
    a.inter = inter;
    a.n = (uint32_t)((int64_t)rows * (inter / 16));
    a.units = FastDiv(inter / 16);
    a.rule = scale_rule;
    a.perm_src = perm_src_d;
    a.codes = codes_d;
    a.sf = sf_d;
    a.layout = sf_layout;
    a.dgu = dgate_up_d;
    const int es = elem_bytes(dtype);
    const bool vec = rows_vec(ds_d, (int64_t)inter * es, rows > 1 ? stride * es : 0);
    return launch(swiglu_back_kernel_for(dtype, vec), dim3(blocks_for((int64_t)rows * (inter / 16), 256, 8)),
                  dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), true, a);
}

moe_status moe_selftest_group_wait(uint32_t* words_d, uint64_t limit_ns, moe_stream_t stream)
{
    const NvtxRange nvtx_range("moe_selftest_group_wait");
    if (!words_d || !elem_aligned(words_d, 4) || limit_ns == 0 || limit_ns > kWaitLimitNs)
        return MOE_ERR_INVALID;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint32_t words[2] = {};
    if (cudaMemsetAsync(words_d, 0, sizeof words, s) != cudaSuccess) return MOE_ERR_CUDA;
    group_wait_probe_kernel<<<1, 256, 0, s>>>(words_d, words_d + 1, limit_ns);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyAsync(words, words_d, sizeof words, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return MOE_ERR_CUDA;
    return words[0] == MOE_DEV_WAIT_TIMEOUT && words[1] == 0xF0u ? MOE_ERR_TIMEOUT : MOE_OK;
}

}  // extern "C"
