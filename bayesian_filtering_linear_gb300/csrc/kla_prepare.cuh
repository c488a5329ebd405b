// Dynamic shared memory above what a kernel may have by default.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace kla {

constexpr int kMaxDevices = 256;
constexpr size_t kMaxSmem = 227 * 1024;  // a block's shared memory at most

// Raise kernel `Kernel`'s dynamic shared-memory limit to `smem_max` — the
// most any launch of that instantiation asks for — once per device. The limit
// belongs to the kernel and not to a launch: set to each call's own size, it
// could be lowered by another thread's call before the launch.
template <auto Kernel>
cudaError_t prepare_kernel(size_t smem_max) {
  static std::atomic<int> done[kMaxDevices];  // one set per kernel instantiation
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_max)) != cudaSuccess)
    return e;
  done[dev].store(1, std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace kla
