// sv_launch.cuh -- attributes of kernels that want more shared memory than the default.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace sv {

// Lets `kernel` have `bytes` of dynamic shared memory, with the largest carveout, on the current device.  Asked of the
// runtime when a device first sees the kernel or a larger size: a call costs the host about a microsecond.
template <typename Kernel>
cudaError_t allow_shared(Kernel *kernel, int bytes, std::atomic<int> (&allowed)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 64;
    if (known && allowed[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e == cudaSuccess && known) allowed[dev].store(bytes, std::memory_order_relaxed);
    return e;
}

}  // namespace sv
