// sv_launch.cuh -- attributes of kernels that want more shared memory than the default.
#pragma once

#include <atomic>
#include <mutex>

#include <cuda_runtime.h>

namespace sv {

// Held while an attribute is set and noted.
inline std::mutex allow_shared_lock;

// Lets `kernel` have `bytes` of dynamic shared memory at least, with the largest carveout, on the current device.  Asked of
// the runtime when a device first sees the kernel or a larger size: a call costs the host about a microsecond.  The limit never
// falls: threads that come with different sizes set and note them one after the other, so that `allowed` is what was set.
template <typename Kernel>
cudaError_t allow_shared(Kernel *kernel, int bytes, std::atomic<int> (&allowed)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;  // (no machine has as many)
    if (allowed[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    std::lock_guard<std::mutex> hold(allow_shared_lock);
    if (allowed[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e == cudaSuccess) allowed[dev].store(bytes, std::memory_order_release);
    return e;
}

}  // namespace sv
