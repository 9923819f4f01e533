// Internal launchers of the operators around the LM head (not part of the public
// ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

// ---- scores of logits (eas_score.cu) ----
constexpr int kMaxTop = 64;       // EAS_MAX_TOP
constexpr int kMaxTokens = 128;   // EAS_MAX_TOKENS
struct ScoreFwdArgs {
  const void* x;          // [N] rows of V logits, ld elements apart
  long long ld;
  const int* tokens;      // [N][M]; -1: none
  const uint8_t* mask;    // [N] or null: every row active
  long long N;
  int V, M, k;
  float scale, c;         // c = scale log2 e
  float* logprob;         // [N][M]
  float* entropy;         // [N]
  float* lse;             // [N]
  float* top;             // [N][k]
  int* ids;               // [N][k]
  DevStatus* status;      // or null
  int split;              // CTAs a row (set by the launcher)
};
cudaError_t launch_score_fwd(const ScoreFwdArgs& a, int is_bf16, int num_sms, cudaStream_t s);

struct ScoreBwdArgs {
  const void* x;
  long long ld;
  const int* tokens;
  const uint8_t* mask;
  const float* g_logprob; // [N][M]
  const float* g_entropy; // [N] or null: zero
  const float* lse;       // [N]
  const float* entropy;   // [N]
  void* dx;               // [N] rows, ld_dx apart; may be x itself
  long long ld_dx;
  long long N;
  int V, M;
  float scale;
  DevStatus* status;
  int split;
};
cudaError_t launch_score_bwd(const ScoreBwdArgs& a, int is_bf16, int num_sms, cudaStream_t s);

// ---- orthogonalised update (eas_muon.cu) ----
constexpr int kMuonSteps = 32;    // EAS_MAX_MUON_STEPS
struct MuonPlan {         // places in the workspace, in bytes from its start
  size_t far_lo;          // of small matrices, all they take: lo that shared memory has no room for
  size_t sync, sync_words;   // from here on: of larger ones
  size_t partial;         // double [L][chunks]
  size_t x[4];            // X's two pairs: hi, lo, hi, lo (fp16)
  size_t gram, poly;
  size_t parts;           // float, of the tiles of A that are computed in parts
  size_t total;
  long long ldx, lda;     // row pitches in elements
  long long chunk, chunks;
  long long split;        // parts of a tile of A
};
MuonPlan muon_plan(long long L, long long rows, long long cols);
struct MuonPair {
  __half *hi, *lo;
};
struct MuonArgs {
  const void* grad;       // [L][rows][cols]
  const void* mom;        // or null
  void* new_mom;          // may be mom
  int mom_bf16;
  int rows, cols, L;
  int n, m, tall;         // X [n][m], n <= m; tall: the transpose of what came
  float beta, rest;       // rest = 1 - beta
  int nesterov;
  float eps, scale;
  const float* coeffs;    // host, [steps][3]
  float small_coeffs[3 * kMuonSteps];   // the same, for the kernel of small matrices
  int steps;
  __nv_bfloat16* out;     // [L][rows][cols]
  double* partial;
  int chunk, chunks;
  MuonPair x[2];
  __half* gram;           // A
  __half* poly;           // B
  float* parts;           // of A's tiles
  uint8_t* far_lo;        // of small matrices
  long long split;
  long long ldx, lda;
  int* sync;              // counters of the products, zero at their start
  long long sync_words;
  DevStatus* status;
  long long budget;       // clocks a wait may take
};
typedef CUresult (*MapEncoder)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
cudaError_t launch_muon(const MuonArgs& a, int grad_bf16, MapEncoder enc, int num_sms, cudaStream_t s);

}  // namespace eas
