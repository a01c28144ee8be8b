// Launching the kernels of attention over a paged cache.
#pragma once

#include <atomic>

#include "attn_common.cuh"

namespace kda {
namespace attn {

// Query rows of an item for `all` rows of a sequence and key head, keys of a unit (its power of two), workers on an SM, and the
// launch, of the kernel for fp32 data and of that for bf16.
int fma_rows(int all);
int fma_unit_shift(const Args &a);
int fma_workers(const Args &a);
cudaError_t launch_attn_fma(const Args &a, cudaStream_t stream);
int mma_rows(int all, int D);
int mma_unit_shift(const Args &a);
int mma_workers(const Args &a);
cudaError_t launch_attn_mma(const Args &a, cudaStream_t stream);

// Launches a kernel of kSmem bytes of shared memory with TEAM warps for each worker.
template <auto kernel, int kSmem, int TEAM>
cudaError_t launch_kernel(const Args &a, cudaStream_t stream) {
    static std::atomic<bool> ready[64];  // per device, of this kernel
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
    }
    kernel<<<a.workers / (kWarps / TEAM), kThreads, kSmem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace kda
