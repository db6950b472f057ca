// pa_device.h -- what a kernel has to be allowed on each device (internal to
// the library).
#pragma once

#include <cuda_runtime_api.h>
#include <stdint.h>

#include <atomic>

namespace pa {

// Lets `kern` take `bytes` of dynamic shared memory on the current device.  The
// limit belongs to the kernel on one device, so `done` (zero at first, one for
// each kernel) keeps a bit for each; devices past its bits are told every time.
// Threads that meet here set the same value twice at worst.
inline cudaError_t allow_shared_memory(const void* kern, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Lets `kern` run in clusters of up to 16 CTAs on the current device; `done` as above.
inline cudaError_t allow_wide_clusters(const void* kern, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace pa
