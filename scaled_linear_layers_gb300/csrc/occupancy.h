// Host helpers: blocks of a kernel that fit one SM, and clusters that fit the
// device, asked once per kernel and device (a persistent kernel sizes its grid
// with them).
#pragma once

#include <atomic>
#include <cuda_runtime.h>

namespace fp8 {

template <auto KERNEL>
cudaError_t blocks_per_sm(int threads, int *out) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < 64;
    int n = cached ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, threads, 0);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        if (cached) known[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return cudaSuccess;
}

// Clusters of `ctas` blocks of a kernel (which takes up to `smem` bytes of
// dynamic shared memory, allowed here) that run at the same time.
template <auto KERNEL>
cudaError_t clusters_resident(int ctas, int threads, size_t smem, int *out) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < 64;
    int n = cached ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        if (cached) known[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return cudaSuccess;
}

}  // namespace fp8
