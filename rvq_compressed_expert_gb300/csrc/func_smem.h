// Dynamic shared memory of kernels that need more than the default (host side).
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace wm {

// Devices the per-device host caches track (ordinals past it are served uncached).
constexpr int kMaxDevices = 64;

// The dynamic shared memory a kernel may ask for is an attribute of the kernel on each
// device: it is set on the current device the first time a launcher needs `bytes` there
// (a cheap driver call; the cache only avoids repeating it).  One SmemAttr per kernel.
struct SmemAttr {
    std::atomic<int> bytes[kMaxDevices] = {};
    std::mutex raising;
};
// Calls of two host threads may need different sizes of one kernel: the attribute is only ever raised, by
// one thread at a time, so that it never falls below what the cache says or a launch on its way needs.
inline cudaError_t ensure_smem(SmemAttr &a, const void *kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && a.bytes[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    const std::lock_guard<std::mutex> one(a.raising);
    if (cached && a.bytes[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && cached) a.bytes[dev].store(bytes, std::memory_order_release);
    return e;
}

} // namespace wm
