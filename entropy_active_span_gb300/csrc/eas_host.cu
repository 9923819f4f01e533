// Errors, device properties, event tracing and the entry points that belong to no
// operator (declared in include/eas.h).
#include "eas_host.h"

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <deque>
#include <mutex>

#include "eas_device.cuh"
#include "eas_kernels.h"

using namespace eas;

namespace {

thread_local char g_err[512] = "";

const char* const kTraceNames[kTrCount] = {
    "spans_build", "rowmap", "gather_rows", "fwd_gemm_tc", "combine", "zero_rows",
    "dlogits_gemm_tc", "dproj_gemm_tc", "unused", "fwd_gemm_simt",
    "dlogits_gemm_simt", "dhidden_gemm_simt", "dweight_gemm_simt", "memset",
    "bwd_chunk_gemm_tc", "dlogits_gemm_tc_e4m3",
    "rmsnorm_fwd", "rmsnorm_bwd", "rmsnorm_dweight", "embed_fwd", "embed_sort", "embed_bwd",
    "grad_norm", "clip_grad_norm", "token_logprobs_fwd", "token_logprobs_bwd",
    "orthogonalize"};

}  // namespace

namespace eas {

eas_status fail(eas_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return s;
}

eas_status cuda_fail(cudaError_t e, const char* what) {
  return fail(EAS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Replaces this thread's eas_last_error() message.
void set_last_error(const char* msg) { snprintf(g_err, sizeof(g_err), "%s", msg); }

eas_status device_info(DevInfo* out) {
  static std::mutex mu;
  static DevInfo cache[64];
  static bool have[64] = {};
  int dev = 0;
  EAS_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(EAS_ERR_UNSUPPORTED, "device ordinal %d", dev);
  std::lock_guard<std::mutex> lk(mu);
  if (!have[dev]) {
    DevInfo d;
    EAS_CUDA(cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev), "sm count");
    EAS_CUDA(cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev), "cc");
    EAS_CUDA(cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev), "cc");
    cache[dev] = d;
    have[dev] = true;
  }
  *out = cache[dev];
  if (out->major != 10 || out->minor != 3)
    return fail(EAS_ERR_UNSUPPORTED, "built for sm_103a; device is sm_%d%d", out->major,
                out->minor);
  return EAS_OK;
}

struct TraceRec {
  int kind;
  cudaEvent_t a, b;
};

namespace {

std::mutex g_trace_mu;
std::atomic<bool> g_trace_on{false};   // read unlocked on every launch
std::deque<TraceRec> g_trace_pool;    // events are created once and reused; a deque
                                      // keeps records in place as it grows
size_t g_trace_used = 0;

}  // namespace

Trace::Trace(int kind, cudaStream_t s) : s_(s) {
  if (!g_trace_on.load(std::memory_order_relaxed)) return;
  std::lock_guard<std::mutex> lk(g_trace_mu);
  if (!g_trace_on.load(std::memory_order_relaxed)) return;
  if (g_trace_used == g_trace_pool.size()) {
    TraceRec r{kind, nullptr, nullptr};
    if (cudaEventCreate(&r.a) != cudaSuccess) return;
    if (cudaEventCreate(&r.b) != cudaSuccess) {
      cudaEventDestroy(r.a);
      return;
    }
    g_trace_pool.push_back(r);
  }
  rec_ = &g_trace_pool[g_trace_used++];
  rec_->kind = kind;
  cudaEventRecord(rec_->a, s_);
}

Trace::~Trace() {
  if (rec_) cudaEventRecord(rec_->b, s_);
}

}  // namespace eas

extern "C" {

eas_status eas_read_device_status(const void* ws, void* stream) {
  if (!ws) return fail(EAS_ERR_INVALID_ARG, "null workspace");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DevStatus h;
  EAS_CUDA(cudaMemcpyAsync(&h, ws, sizeof(h), cudaMemcpyDeviceToHost, s), "read status");
  EAS_CUDA(cudaStreamSynchronize(s), "stream sync");
  if (h.code != 0)
    return fail(static_cast<eas_status>(h.code), "device status %d (where %d, info %d)", h.code,
                h.where, h.info);
  return EAS_OK;
}

void eas_trace_enable(int32_t on) {
  std::lock_guard<std::mutex> lk(g_trace_mu);
  g_trace_on.store(on != 0, std::memory_order_relaxed);
  if (on != 0) g_trace_used = 0;
}

int32_t eas_trace_read(int32_t* kinds, float* ms, int32_t cap) {
  std::lock_guard<std::mutex> lk(g_trace_mu);
  const int32_t n = static_cast<int32_t>(g_trace_used);
  for (int32_t i = 0; i < n && i < cap; ++i) {
    const TraceRec& r = g_trace_pool[i];
    float t = -1.f;
    if (cudaEventSynchronize(r.b) != cudaSuccess || cudaEventElapsedTime(&t, r.a, r.b) != cudaSuccess)
      t = -1.f;
    if (kinds) kinds[i] = r.kind;
    if (ms) ms[i] = t;
  }
  return n;
}

const char* eas_kernel_name(int32_t kind) {
  return (kind >= 0 && kind < kTrCount) ? kTraceNames[kind] : "unknown";
}

const char* eas_last_error(void) { return g_err; }

const char* eas_status_string(eas_status s) {
  switch (s) {
    case EAS_OK: return "EAS_OK";
    case EAS_ERR_INVALID_ARG: return "EAS_ERR_INVALID_ARG";
    case EAS_ERR_INVALID_SPANS: return "EAS_ERR_INVALID_SPANS";
    case EAS_ERR_UNSUPPORTED: return "EAS_ERR_UNSUPPORTED";
    case EAS_ERR_WORKSPACE: return "EAS_ERR_WORKSPACE";
    case EAS_ERR_CUDA: return "EAS_ERR_CUDA";
    case EAS_ERR_TIMEOUT: return "EAS_ERR_TIMEOUT";
    case EAS_ERR_SPAN_CAPACITY: return "EAS_ERR_SPAN_CAPACITY";
    case EAS_ERR_INVALID_LAYOUT: return "EAS_ERR_INVALID_LAYOUT";
  }
  return "EAS_UNKNOWN";
}

int32_t eas_version(void) { return 100; }

}  // extern "C"
