// Launches of the operators around the LM head: shared memory, and launches that
// overlap (programmatic dependent launch).
#pragma once

#include <atomic>
#include <cuda_runtime.h>
#include <stdint.h>

namespace eas {

// Lets the next launch on the stream begin, if it was launched to overlap
// (launch_overlapped); what this grid writes is not visible to it yet.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Waits until the launch before has ended and its writes are visible.
__device__ __forceinline__ void wait_for_launch_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches a kernel that may begin before the launch in front of it on the
// stream has ended; it calls wait_for_launch_before() ahead of its first use of
// that launch's results, or at its end.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t s, A... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

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
