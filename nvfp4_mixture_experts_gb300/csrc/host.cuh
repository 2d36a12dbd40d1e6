// Host-side helpers of the C ABI's translation units: NVTX ranges, tensor-map encoding, kernel
// launches with their attributes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <mutex>

#include "kernels.cuh"

namespace {

// ---------------------------------------------------------------- NVTX ranges
// Every C-ABI call that launches work opens a range named after itself in the "nvfp4moe"
// domain (host-side; a profiler attributes the call's launches to it).  With no tool
// attached an NVTX call returns at once.
struct NvtxRange {
    explicit NvtxRange(const char* name)
    {
        static const nvtxDomainHandle_t domain = nvtxDomainCreateA("nvfp4moe");
        nvtxEventAttributes_t a = {};
        a.version = NVTX_VERSION;
        a.size = NVTX_EVENT_ATTRIB_STRUCT_SIZE;
        a.messageType = NVTX_MESSAGE_TYPE_ASCII;
        a.message.ascii = name;
        nvtxDomainRangePushEx(domain, &a);
        dom = domain;
    }
    ~NvtxRange() { nvtxDomainRangePop(dom); }
    nvtxDomainHandle_t dom;
};

// ---------------------------------------------------------------- driver entry point
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn()
{
    // A host thread that has made no runtime call that needs a context has none, and encoding, a
    // driver call, does not make it current; setting the thread's device does.
    thread_local const bool context = [] {
        int dev = 0;
        return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
    }();
    if (!context) return nullptr;
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2-D tensor map over rows of row_bytes (dims in elements of dtype).
inline bool make_tmap(CUtensorMap* m, const void* base, CUtensorMapDataType dtype,
                      uint64_t inner, uint64_t rows, uint64_t row_bytes, uint32_t box_inner,
                      uint32_t box_rows, CUtensorMapSwizzle swz)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc || rows == 0) return false;
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {box_inner, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, dtype, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D tensor map: matrices of rows of row_bytes, row_bytes * rows apart; boxes of one matrix.
inline bool make_tmap_3d(CUtensorMap* m, const void* base, CUtensorMapDataType dtype,
                         uint64_t inner, uint64_t rows, uint64_t matrices, uint64_t row_bytes,
                         uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swz)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc || rows == 0 || matrices == 0) return false;
    const cuuint64_t dims[3] = {inner, rows, matrices};
    const cuuint64_t strides[2] = {row_bytes, row_bytes * rows};
    const cuuint32_t box[3] = {box_inner, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, dtype, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

inline int ceil_div(int a, int b) { return moe::div_up(a, b); }

// Whether a runtime call succeeded; the error of one that did not is reported by its caller, and taken
// from the thread's last error, where the check of a later launch would find it.
inline bool taken(cudaError_t e)
{
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess;
}

inline moe_status check_launch()
{
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Launches a kernel, with programmatic dependent launch when pdl is set (the forward's
// chain: each kernel may start while its predecessor finishes; see pdl_wait()).
template <typename... KArgs, typename... Args>
moe_status launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                  bool pdl, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return taken(cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...)) ? MOE_OK : MOE_ERR_CUDA;
}

// A launch whose blocks wait on one another (the fused W4A16 GEMV's down items wait for gate_up
// tiles of other blocks): cooperative, so that every block is resident at once or the launch
// fails.
template <typename... KArgs, typename... Args>
moe_status launch_coop(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t s, bool pdl, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return taken(cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...)) ? MOE_OK : MOE_ERR_CUDA;
}

// As launch, for a kernel whose blocks run as clusters of `blocks`.
template <typename... KArgs, typename... Args>
moe_status launch_cluster(void (*kern)(KArgs...), int blocks, dim3 grid, dim3 block, size_t smem,
                          cudaStream_t s, bool pdl, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return taken(cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...)) ? MOE_OK : MOE_ERR_CUDA;
}

// As launch, for a kernel whose blocks run as CTA pairs.
template <typename... KArgs, typename... Args>
moe_status launch_pairs(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                        bool pdl, Args... args)
{
    return launch_cluster(kern, 2, grid, block, smem, s, pdl, args...);
}

}  // namespace
