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

// How many clusters of `size` CTAs (16 at most) of `kern` the current device holds
// at once, `cfg` being their launch but for its grid; `known` keeps the answers, one
// for each device and size.  0 where the question fails.
inline int clusters_at_once(const void* kern, cudaLaunchConfig_t cfg, int size,
                            std::atomic<uint16_t> (&known)[64][17]) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool kept = dev >= 0 && dev < 64;
    const uint16_t before = kept ? known[dev][size].load(std::memory_order_relaxed) : 0;
    if (before) return before - 1;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(size);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(unsigned(size));
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (n > 65534) n = 65534;
    if (kept) known[dev][size].store(uint16_t(n + 1), std::memory_order_relaxed);
    return n;
}

}  // namespace pa
