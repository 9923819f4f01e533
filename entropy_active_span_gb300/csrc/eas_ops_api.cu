// C ABI of the operators around the LM head (declared in include/eas.h): argument
// checks and the launch sequence of each call, as in eas_api.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>
#include <vector>

#include "eas_device.cuh"
#include "eas_host.h"
#include "eas_ops.h"

using namespace eas;

namespace {

// A buffer of a call.  `shared`: a written one may replace, whole, a read one that
// is also marked so.
struct Buf {
  const void* p;
  size_t n;
  bool shared = false;
};

// Whether no written buffer shares a byte with another buffer (null shares none).
bool disjoint(std::initializer_list<Buf> written, std::initializer_list<Buf> read) {
  auto overlap = [](const Buf& a, const Buf& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && a.n && b.n && x < y + b.n && y < x + a.n;
  };
  for (const Buf* w = written.begin(); w != written.end(); ++w) {
    for (const Buf* v = w + 1; v != written.end(); ++v)
      if (overlap(*w, *v)) return false;
    for (const Buf& r : read)
      if (!(w->shared && r.shared && w->p == r.p && w->n == r.n) && overlap(*w, r)) return false;
  }
  return true;
}

eas_status overlap_error() { return fail(EAS_ERR_INVALID_ARG, "an output or the workspace overlaps another buffer"); }

// Shape and type of the row operators: any H (odd ones keep their vectors on
// 16-byte boundaries in memory).
eas_status check_rows(long long R, long long H, eas_dtype dt) {
  if (R < 0 || R > 0x7fffff00LL) return fail(EAS_ERR_INVALID_ARG, "rows=%lld out of range", R);
  if (H < 1 || H > (1LL << 20)) return fail(EAS_ERR_INVALID_ARG, "H=%lld out of range", H);
  if (dt != EAS_BF16 && dt != EAS_FP32) return fail(EAS_ERR_INVALID_ARG, "dtype %d", (int)dt);
  return EAS_OK;
}

size_t norm_bwd_rstd_offset(long long R, long long H) {
  return align_up(sizeof(DevStatus)) + align_up(4 * static_cast<size_t>(rmsnorm_bwd_partials(R, H)) * static_cast<size_t>(H));
}

eas_status check_embed(long long T, long long H, long long V, eas_dtype dt, float scale) {
  eas_status st = check_rows(T, H, dt);
  if (st != EAS_OK) return st;
  if (V < 1 || V > 0x7fffff00LL) return fail(EAS_ERR_INVALID_ARG, "V=%lld out of range", V);
  if (!std::isfinite(scale)) return fail(EAS_ERR_INVALID_ARG, "scale must be finite");
  return EAS_OK;
}

}  // namespace

extern "C" {

eas_status eas_rmsnorm_fwd(const void* x, const void* residual, const void* weight,
                           const uint8_t* mask, int64_t R, int64_t H, eas_dtype dtype, float eps,
                           void* sum_out, void* y, uint8_t* y_e4m3, float* y_scale, void* stream) {
  eas_status st = check_rows(R, H, dtype);
  if (st != EAS_OK) return st;
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(EAS_ERR_INVALID_ARG, "eps must be positive");
  if (!weight || (R > 0 && !x)) return fail(EAS_ERR_INVALID_ARG, "null pointer");
  if ((y_e4m3 == nullptr) != (y_scale == nullptr))
    return fail(EAS_ERR_INVALID_ARG, "y_e4m3 and y_scale come together");
  if (sum_out && !residual) return fail(EAS_ERR_INVALID_ARG, "sum_out needs a residual");
  if (R > 0 && !y && !y_e4m3 && !sum_out) return fail(EAS_ERR_INVALID_ARG, "no output");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum_out, 16) ||
      !aligned(y, 16) || !aligned(y_e4m3, 16) || !aligned(y_scale, 4))
    return fail(EAS_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  const size_t codes = static_cast<size_t>(R) * static_cast<size_t>(H), rows = codes * elem_size(dtype);
  if (!disjoint({{sum_out, rows, true}, {y, rows}, {y_e4m3, codes}, {y_scale, 4 * static_cast<size_t>(R)}},
                {{x, rows, true}, {residual, rows, true}, {weight, static_cast<size_t>(H) * elem_size(dtype)},
                 {mask, static_cast<size_t>(R)}}))
    return overlap_error();
  DevInfo di;
  st = device_info(&di);
  if (st != EAS_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RmsNormFwdArgs a = {x, residual, weight, mask, sum_out, y, y_e4m3, y_scale,
                            R, static_cast<int>(H), eps};
  Trace tr_(kTrNormFwd, s);
  EAS_CUDA(launch_rmsnorm_fwd(a, dtype == EAS_BF16, di.sms, s), "rmsnorm_fwd");
  return EAS_OK;
}

size_t eas_rmsnorm_bwd_workspace_size(int64_t R, int64_t H) {
  if (R < 0 || H < 1) return 0;
  return norm_bwd_rstd_offset(R, H) + align_up(4 * static_cast<size_t>(R));
}

eas_status eas_rmsnorm_bwd(const void* dy, const void* sum, const void* weight, const void* ds,
                           const uint8_t* mask, int64_t R, int64_t H, eas_dtype dtype, float eps,
                           void* dx, float* dweight, void* ws, size_t ws_bytes, void* stream) {
  eas_status st = check_rows(R, H, dtype);
  if (st != EAS_OK) return st;
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(EAS_ERR_INVALID_ARG, "eps must be positive");
  if (!weight || !dweight || !ws || (R > 0 && (!dy || !sum || !dx)))
    return fail(EAS_ERR_INVALID_ARG, "null pointer");
  if (!aligned(dy, 16) || !aligned(sum, 16) || !aligned(weight, 16) || !aligned(ds, 16) ||
      !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(ws, 256))
    return fail(EAS_ERR_INVALID_ARG, "tensors must be 16-byte and ws 256-byte aligned");
  const size_t need = eas_rmsnorm_bwd_workspace_size(R, H);
  if (ws_bytes < need) return fail(EAS_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, need);
  const size_t row = static_cast<size_t>(H) * elem_size(dtype), rows = static_cast<size_t>(R) * row;
  if (!disjoint({{dx, rows, true}, {dweight, 4 * static_cast<size_t>(H)}, {ws, need}},
                {{dy, rows}, {sum, rows}, {weight, row}, {ds, rows, true}, {mask, static_cast<size_t>(R)}}))
    return overlap_error();
  DevInfo di;
  st = device_info(&di);
  if (st != EAS_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RmsNormBwdArgs a = {dy, sum, weight, ds, mask, dx, at<float>(ws, align_up(sizeof(DevStatus))),
                            at<float>(ws, norm_bwd_rstd_offset(R, H)), R, static_cast<int>(H), eps};
  int n = 0;
  {
    Trace tr_(kTrNormBwd, s);
    EAS_CUDA(launch_rmsnorm_bwd(a, dtype == EAS_BF16, di.sms, &n, s), "rmsnorm_bwd");
  }
  {
    Trace tr_(kTrNormDw, s);
    EAS_CUDA(launch_rmsnorm_dw(a.partial, n, a.H, dweight, static_cast<DevStatus*>(ws), s), "rmsnorm_dweight");
  }
  return EAS_OK;
}

eas_status eas_embed_fwd(const int32_t* ids, const void* table, int64_t T, int64_t H, int64_t V,
                         eas_dtype dtype, float scale, void* out, void* ws, size_t ws_bytes,
                         void* stream) {
  eas_status st = check_embed(T, H, V, dtype, scale);
  if (st != EAS_OK) return st;
  if (!table || (T > 0 && (!ids || !out))) return fail(EAS_ERR_INVALID_ARG, "null pointer");
  if (!aligned(ids, 4) || !aligned(table, 16) || !aligned(out, 16) || !aligned(ws, 16))
    return fail(EAS_ERR_INVALID_ARG, "table, out and ws must be 16-byte aligned");
  if (ws && ws_bytes < sizeof(DevStatus)) return fail(EAS_ERR_WORKSPACE, "workspace too small");
  const size_t row = static_cast<size_t>(H) * elem_size(dtype), n = static_cast<size_t>(T);
  if (!disjoint({{out, row * n}, {ws, sizeof(DevStatus)}}, {{ids, 4 * n}, {table, row * static_cast<size_t>(V)}}))
    return overlap_error();
  DevInfo di;
  st = device_info(&di);
  if (st != EAS_OK) return st;
  if (T == 0 && !ws) return EAS_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const EmbedFwdArgs a = {ids, table, out, T, static_cast<int>(V), static_cast<int>(H), scale,
                          static_cast<DevStatus*>(ws)};
  Trace tr_(kTrEmbedFwd, s);
  EAS_CUDA(launch_embed_fwd(a, dtype == EAS_BF16, di.sms, s), "embed_fwd");
  return EAS_OK;
}

size_t eas_embed_bwd_workspace_size(int64_t T, int64_t H, int64_t V) {
  if (T < 0 || H < 1 || V < 1) return 0;
  return align_up(sizeof(DevStatus)) + embed_bwd_plan(T, H, V).total;
}

eas_status eas_embed_bwd(const int32_t* ids, const void* dout, int64_t T, int64_t H, int64_t V,
                         eas_dtype dtype, float scale, int32_t accumulate, float* dweight,
                         void* ws, size_t ws_bytes, void* stream) {
  eas_status st = check_embed(T, H, V, dtype, scale);
  if (st != EAS_OK) return st;
  if (accumulate != 0 && accumulate != 1) return fail(EAS_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  if (!dweight || !ws || (T > 0 && (!ids || !dout))) return fail(EAS_ERR_INVALID_ARG, "null pointer");
  if (!aligned(ids, 4) || !aligned(dout, 16) || !aligned(dweight, 16) || !aligned(ws, 256))
    return fail(EAS_ERR_INVALID_ARG, "dout and dweight must be 16-byte and ws 256-byte aligned");
  const size_t need = eas_embed_bwd_workspace_size(T, H, V);
  if (ws_bytes < need) return fail(EAS_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, need);
  const size_t n = static_cast<size_t>(T), h = static_cast<size_t>(H);
  if (!disjoint({{dweight, 4 * static_cast<size_t>(V) * h}, {ws, need}}, {{ids, 4 * n}, {dout, n * h * elem_size(dtype)}}))
    return overlap_error();
  DevInfo di;
  st = device_info(&di);
  if (st != EAS_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const EmbedBwdArgs a = {ids, dout, dweight, T, static_cast<int>(V), static_cast<int>(H), scale,
                          accumulate, at<char>(ws, align_up(sizeof(DevStatus))),
                          static_cast<DevStatus*>(ws)};
  if (embed_bwd_sorts(T)) {
    Trace tr_(kTrEmbedSort, s);
    EAS_CUDA(launch_embed_sort(a, s), "embed_sort");
  }
  Trace tr_(kTrEmbedBwd, s);
  EAS_CUDA(launch_embed_bwd(a, dtype == EAS_BF16, di.sms, s), "embed_bwd");
  return EAS_OK;
}

size_t eas_clip_grad_norm_workspace_size(int32_t n) {
  if (n < 0) return 0;
  return align_up(sizeof(DevStatus)) + clip_workspace_bytes(n);
}

eas_status eas_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels,
                              const int32_t* dtypes, const int32_t* out_dtypes, int32_t n,
                              float max_norm, float* norm, void* ws, size_t ws_bytes,
                              void* stream) {
  if (n < 0 || n > (1 << 20)) return fail(EAS_ERR_INVALID_ARG, "n=%d out of range", n);
  if (!norm || !ws || (n > 0 && (!grads || !numels || !dtypes)) || (n > 0 && outs && !out_dtypes))
    return fail(EAS_ERR_INVALID_ARG, "null pointer");
  if (outs && !(max_norm >= 0.f)) return fail(EAS_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (!aligned(norm, 4) || !aligned(ws, 256))
    return fail(EAS_ERR_INVALID_ARG, "ws must be 256-byte aligned");
  const size_t need = eas_clip_grad_norm_workspace_size(n);
  if (ws_bytes < need) return fail(EAS_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, need);
  try {
    std::vector<ClipTensor> list(static_cast<size_t>(n));
    // every buffer that is written, and every one that is read, by address (tensor
    // -1: the norm and the workspace)
    struct Range {
      uintptr_t lo, hi;
      int tensor;
      bool written;
    };
    std::vector<Range> ranges;
    ranges.reserve(2 * static_cast<size_t>(n) + 2);
    const uintptr_t np = reinterpret_cast<uintptr_t>(norm), wp = reinterpret_cast<uintptr_t>(ws);
    ranges.push_back({np, np + sizeof(float), -1, true});
    ranges.push_back({wp, wp + need, -1, true});
    for (int i = 0; i < n; ++i) {
      ClipTensor& t = list[i];
      t.in = grads[i];
      t.out = outs ? outs[i] : nullptr;
      t.numel = numels[i];
      const int id = dtypes[i], od = outs ? out_dtypes[i] : id;
      if ((id != EAS_BF16 && id != EAS_FP32) || (od != EAS_BF16 && od != EAS_FP32))
        return fail(EAS_ERR_INVALID_ARG, "tensor %d: dtype %d / %d", i, id, od);
      t.in_bf16 = id == EAS_BF16;
      t.out_bf16 = od == EAS_BF16;
      if (t.numel < 0 || t.numel > (1LL << 40))
        return fail(EAS_ERR_INVALID_ARG, "tensor %d: numel %lld", i, t.numel);
      if (t.numel == 0) continue;
      if (!t.in || (outs && !t.out)) return fail(EAS_ERR_INVALID_ARG, "tensor %d: null pointer", i);
      const size_t ie = t.in_bf16 ? 2 : 4, oe = t.out_bf16 ? 2 : 4;
      if (!aligned(t.in, ie) || (outs && !aligned(t.out, oe)))
        return fail(EAS_ERR_INVALID_ARG, "tensor %d: not aligned to its element", i);
      const uintptr_t ip = reinterpret_cast<uintptr_t>(t.in), op = reinterpret_cast<uintptr_t>(t.out);
      if (ip == op && ie != oe)
        return fail(EAS_ERR_INVALID_ARG, "tensor %d: in place with another dtype", i);
      if (outs) ranges.push_back({op, op + oe * static_cast<size_t>(t.numel), i, true});
      if (ip != op) ranges.push_back({ip, ip + ie * static_cast<size_t>(t.numel), i, false});
    }
    // no written buffer may share a byte with another entry's, with its own input
    // or with the norm or the workspace
    std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t end = 0, written_end = 0;
    for (const Range& r : ranges) {
      if (r.lo < (r.written ? end : written_end))
        return r.tensor < 0 ? overlap_error()
                            : fail(EAS_ERR_INVALID_ARG, "tensor %d overlaps another buffer", r.tensor);
      end = r.hi > end ? r.hi : end;
      if (r.written) written_end = r.hi > written_end ? r.hi : written_end;
    }
    DevInfo di;
    eas_status st = device_info(&di);
    if (st != EAS_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Trace tr_(outs ? kTrGradClip : kTrGradNorm, s);
    EAS_CUDA(launch_clip_grad_norm(list.data(), n, outs != nullptr, max_norm,
                                   at<double>(ws, align_up(sizeof(DevStatus))), norm,
                                   static_cast<DevStatus*>(ws), di.sms, s),
             "clip_grad_norm");
    return EAS_OK;
  } catch (const std::bad_alloc&) {
    return fail(EAS_ERR_CUDA, "out of host memory");
  }
}

}  // extern "C"
