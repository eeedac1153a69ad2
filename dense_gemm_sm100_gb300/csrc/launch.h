// Launch helpers of the router, the 8-bit conversions and the orthogonalised
// update: programmatic stream serialisation, and kernels loaded before use.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <type_traits>

namespace dg {

extern PFN_cuCtxGetId_v12000 g_context_id;  // looked up by gemm_create

// Loads a kernel in the current context and allows it `smem` bytes of dynamic
// shared memory, the first time it is used there: the call may be captured in a
// graph, and loading is no part of that.  Remembered is the last context of every
// device; contexts that take turns on one cost a few microseconds at each change.
template <auto Kernel>
inline cudaError_t kernel_ready(size_t smem)
{
    static std::atomic<unsigned long long> ready[64];  // a context's id + 1
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    unsigned long long id = 0;
    const bool known = dev < 64 && g_context_id(nullptr, &id) == CUDA_SUCCESS;
    if (known && ready[dev].load(std::memory_order_acquire) == id + 1) return cudaSuccess;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // of this thread, for these calls
    if ((e = cudaThreadExchangeStreamCaptureMode(&mode)) != cudaSuccess) return e;
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, Kernel);
    if (e == cudaSuccess && smem + attr.sharedSizeBytes > 48 * 1024)  // with the kernel's static shared memory
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess && known) ready[dev].store(id + 1, std::memory_order_release);
    return e;
}

// The grid of a kernel whose CTAs take one unit after another (max_ctas 0: no cap).
inline int capped(int64_t grid, int max_ctas)
{
    return static_cast<int>(max_ctas > 0 ? std::min<int64_t>(grid, max_ctas) : grid);
}

// cluster: CTAs of a cluster (1: none).
template <typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(Args...), int grid, int threads, size_t smem, cudaStream_t stream,
                              int cluster, const std::common_type_t<Args> &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dg
