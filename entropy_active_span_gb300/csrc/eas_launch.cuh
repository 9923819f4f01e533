// Host-side launch helpers of the operators around the LM head.
#pragma once

#include <atomic>
#include <cuda_runtime.h>
#include <stdint.h>

namespace eas {

// Lets kKernel's launches have up to `bytes` of dynamic shared memory: opted into
// once per device and instantiation (one bit per device ordinal; a repeated opt-in
// is harmless).  The limit belongs to the kernel on the device, not to the thread
// that sets it, so `bytes` is the most that any launch of kKernel takes and always
// the same: set to each launch's own size, it could be lowered by another host
// thread between this thread's opt-in and its launch, which then fails.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (bit != 0 && (configured.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace eas
