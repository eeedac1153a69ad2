// Launch helpers of the router, the 8-bit conversions and the orthogonalised
// update: programmatic stream serialisation, and kernels loaded before use.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <type_traits>

namespace dg {

// Loads a kernel on the current device and allows it `smem` bytes of dynamic
// shared memory, the first time it is used there: the call may be captured in a
// graph, and loading is no part of that.
template <auto Kernel>
inline cudaError_t kernel_ready(size_t smem)
{
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // of this thread, for these calls
    if ((e = cudaThreadExchangeStreamCaptureMode(&mode)) != cudaSuccess) return e;
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, Kernel);
    if (e == cudaSuccess && smem + attr.sharedSizeBytes > 48 * 1024)  // with the kernel's static shared memory
        e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
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
