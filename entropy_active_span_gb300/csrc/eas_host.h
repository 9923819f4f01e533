// Host side that the C-ABI translation units share: errors, argument helpers,
// device properties and event tracing.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/eas.h"

namespace eas {

// Sets this thread's eas_last_error() message and returns s.
eas_status fail(eas_status s, const char* fmt, ...);
eas_status cuda_fail(cudaError_t e, const char* what);

#define EAS_CUDA(call, what)                  \
  do {                                        \
    cudaError_t e_ = (call);                  \
    if (e_ != cudaSuccess) return cuda_fail(e_, what); \
  } while (0)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t elem_size(eas_dtype dt) { return dt == EAS_BF16 ? 2 : dt == EAS_E4M3 ? 1 : 4; }

inline size_t align_up(size_t x) { return (x + 1023) / 1024 * 1024; }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

struct DevInfo {
  int sms = 0;
  int major = 0, minor = 0;
};

eas_status device_info(DevInfo* out);

// When enabled, every kernel launch of the library is bracketed by a pair of
// CUDA events on its stream, tagged with the kernel's kind; eas_trace_read()
// returns the durations.  Off by default; meant for eager (not captured)
// launches.  Backward tensor-core launches are named by their jobs:
// dlogits_gemm_tc (d-logits of chunk 0), bwd_chunk_gemm_tc (dW and dHidden of
// chunk c-1 with the d-logits of chunk c), dproj_gemm_tc (dW and dHidden of
// the last chunk); the e4m3 backward runs dlogits_gemm_tc_e4m3 (d-logits of a
// chunk) and dproj_gemm_tc (dW and dHidden of that chunk) per chunk.

enum TraceKind : int {
  kTrSpans = 0, kTrRowmap, kTrGather, kTrFwdGemm, kTrCombine, kTrZeroRows,
  kTrDLogitsGemm, kTrDProjGemm, kTrUnused, kTrSimtFwd, kTrSimtDLogits,
  kTrSimtDHidden, kTrSimtDWeight, kTrMemset, kTrBwdChunkGemm, kTrDLogitsFp8Gemm,
  kTrNormFwd, kTrNormBwd, kTrNormDw, kTrEmbedFwd, kTrEmbedSort, kTrEmbedBwd, kTrGradNorm,
  kTrGradClip, kTrCount
};

class Trace {
 public:
  Trace(int kind, cudaStream_t s);
  ~Trace();
  Trace(const Trace&) = delete;
  Trace& operator=(const Trace&) = delete;

 private:
  cudaStream_t s_;
  struct TraceRec* rec_ = nullptr;
};

}  // namespace eas
