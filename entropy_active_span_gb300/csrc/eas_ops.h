// Internal launchers of the operators around the LM head (not part of the public
// ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace eas {

struct DevStatus;

// ---- RMS norm (eas_norm.cu) ----
struct RmsNormFwdArgs {
  const void* x;          // [R][H]
  const void* r;          // residual [R][H] or null
  const void* w;          // [H]
  const uint8_t* mask;    // [R] or null: every row active
  void* s_out;            // x + r [R][H] or null; may be x or r itself
  void* y;                // [R][H] or null
  uint8_t* q;             // e4m3 codes [R][H] or null
  float* scale;           // [R], with q
  long long R;
  int H;
  float eps;
};
cudaError_t launch_rmsnorm_fwd(const RmsNormFwdArgs& a, int is_bf16, int num_sms, cudaStream_t s);

struct RmsNormBwdArgs {
  const void* dy;         // [R][H]
  const void* s;          // [R][H]
  const void* w;          // [H]
  const void* ds;         // [R][H] or null; may be dx itself
  const uint8_t* mask;    // [R] or null
  void* dx;               // [R][H]
  float* partial;         // [rmsnorm_bwd_partials(R, H)][H]
  float* rstd;            // [R], rows too long for the ring
  long long R;
  int H;
  float eps;
};
long long rmsnorm_bwd_partials(long long R, long long H);
// Writes dx and *n_partials rows of partial; launch_rmsnorm_dw sums them.
cudaError_t launch_rmsnorm_bwd(const RmsNormBwdArgs& a, int is_bf16, int num_sms, int* n_partials,
                               cudaStream_t s);
// Also clears the status word.
cudaError_t launch_rmsnorm_dw(const float* partial, int n, int H, float* dw, DevStatus* st,
                              cudaStream_t s);

// ---- embedding (eas_embed.cu) ----
struct EmbedFwdArgs {
  const int* ids;         // [T]; -1: padding
  const void* table;      // [V][H]
  void* out;              // [T][H]
  long long T;
  int V, H;
  float scale;
  DevStatus* status;      // or null
};
cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, int is_bf16, int num_sms, cudaStream_t s);

struct EmbedBwdPlan {     // sizes of the backward's scratch, in bytes from its start
  size_t keys[2], pos[2]; // the sort's two buffers of (id, token)
  size_t hist;            // digit counts of the sort's tiles
  size_t partial;         // sums of the pieces of rows that several workers share
  size_t runs;            // where those rows' tokens start in the sorted list
  size_t total;
  int chunk;              // sorted tokens a worker
};
EmbedBwdPlan embed_bwd_plan(long long T, long long H, long long V);
struct EmbedBwdArgs {
  const int* ids;         // [T]; -1: padding
  const void* dout;       // [T][H]
  float* dw;              // [V][H]
  long long T;
  int V, H;
  float scale;
  int accumulate;         // add to dw; else every row of dw is written
  char* scratch;
  DevStatus* status;
};
// Whether a list is long enough to be sorted; the sort clears the status word,
// and without one launch_embed_bwd does.
bool embed_bwd_sorts(long long T);
cudaError_t launch_embed_sort(const EmbedBwdArgs& a, cudaStream_t s);
cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, int is_bf16, int num_sms, cudaStream_t s);

// ---- gradient norm and clipping (eas_clip.cu) ----
struct ClipTensor {
  const void* in;
  void* out;
  long long numel;
  int in_bf16, out_bf16;
};
size_t clip_workspace_bytes(long long n_tensors);
// The norm, and with `clip` the scaled tensors too; clears the status word.
cudaError_t launch_clip_grad_norm(const ClipTensor* t, int n, bool clip, float max_norm,
                                  double* partial, float* norm, DevStatus* st, int num_sms,
                                  cudaStream_t s);

}  // namespace eas
