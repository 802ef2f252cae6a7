// Host helper: blocks of a kernel that fit one SM, asked once per kernel,
// block size and device (a persistent kernel sizes its grid with it).
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

}  // namespace fp8
