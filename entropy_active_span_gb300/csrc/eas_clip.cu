// Global norm of a list of gradients, and clipping.
//
//   norm = sqrt(sum over every tensor of g^2),
//   c = min(1, max_norm / (norm + 1e-6)),  out = c g   (c = 1: norm not finite).
//
// The list travels as a kernel argument: no table in device memory, no copy,
// and a captured graph holds its own.  Work is cut into chunks of kChunk
// elements over all tensors; a CTA finds a chunk's tensor by bisection.
// Squares are added up in fp32 over the 16 bytes of a load, and those sums in
// fp64 from there on.  Every CTA leaves one fp64 partial sum and whoever needs
// the norm adds the partials in the same order, so results repeat to the bit.
#include "eas_device.cuh"
#include "eas_kernels.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;        // elements a chunk
constexpr int kMaxCtas = 1216;       // partials a launch leaves at most
constexpr int kSmallList = 24;
constexpr int kLargeList = 800;

template <int N>
struct List {
  const void* in[N];
  void* out[N];
  long long numel[N];
  int first[N];                      // chunk at which the tensor starts
  unsigned char kind[N];             // bit 0: in is bf16, bit 1: out is bf16
  int n;
  int n_chunks;
};

template <int N>
__device__ __forceinline__ int tensor_of(const List<N>& l, int chunk) {
  int lo = 0, hi = l.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// Sum of squares of one load.  Where the fp32 squares leave the normal range
// (a gradient over 1e18 or all below 1e-15) they are taken again in fp64.
template <int VEC>
__device__ __forceinline__ double squares(const float (&f)[VEC]) {
  float s = 0.f, m = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    s = fmaf(f[i], f[i], s);
    m = fmaxf(m, fabsf(f[i]));
  }
  if (m != 0.f && !(s > 1e-30f && s < 1e36f)) {
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) d += static_cast<double>(f[i]) * f[i];
    return d;
  }
  return s;
}

// Elements before the first 16-byte boundary at or after p.
template <typename T>
__device__ __forceinline__ int head_of(const T* p) {
  return static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int n) {
  constexpr int VEC = kVec16<T>;
  constexpr int U = 4;
  double acc = 0.0;
  int head = head_of(p);
  if (head > n) head = n;
  const int vecs = (n - head) / VEC;
  const T* v = p + head;
  for (int i = threadIdx.x; i < vecs; i += kThreads * U) {
    Raw<T, VEC> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kThreads < vecs) raw[u] = load_raw<T, VEC>(v + static_cast<long long>(i + u * kThreads) * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kThreads < vecs) {
        float f[VEC];
        widen<T, VEC>(raw[u], f);
        acc += squares<VEC>(f);
      }
  }
  const int tail = head + vecs * VEC;
  for (int i = threadIdx.x; i < head + (n - tail); i += kThreads) {
    const double f = to_f32(p[i < head ? i : tail + (i - head)]);
    acc += f * f;
  }
  return acc;
}

__device__ __forceinline__ double block_sum(double v, double* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v += sm[w];
  return v;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
grad_squares_kernel(const __grid_constant__ List<N> l, double* partial) {
  __shared__ double sm[kThreads / 32];
  double acc = 0.0;
  for (int k = blockIdx.x; k < l.n_chunks; k += gridDim.x) {
    const int t = tensor_of(l, k);
    const long long off = static_cast<long long>(k - l.first[t]) * kChunk;
    const long long left = l.numel[t] - off;
    const int n = static_cast<int>(left < kChunk ? left : kChunk);
    if (l.kind[t] & 1)
      acc += chunk_squares(static_cast<const __nv_bfloat16*>(l.in[t]) + off, n);
    else
      acc += chunk_squares(static_cast<const float*>(l.in[t]) + off, n);
  }
  acc = block_sum(acc, sm);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

__global__ void __launch_bounds__(kThreads)
grad_norm_kernel(const double* partial, int n, float* norm) {
  __shared__ double sm[kThreads / 32];
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += partial[i];
  acc = block_sum(acc, sm);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(acc));
}

template <typename I, typename O>
__device__ __forceinline__ void scale_chunk(const I* in, O* out, int n, float c) {
  // vectors of 4 elements: 16 bytes of fp32, 8 of bf16
  constexpr int VEC = 4;
  int head = head_of(in);
  if (head > n) head = n;
  const bool vec = (reinterpret_cast<uintptr_t>(out + head) % (VEC * sizeof(O))) == 0;
  const int vecs = vec ? (n - head) / VEC : 0;
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    float f[VEC];
    if constexpr (sizeof(I) == 4) {
      const float4 q = *reinterpret_cast<const float4*>(in + head + i * VEC);
      f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(in + head + i * VEC);
      f[0] = bf16_lo(q.x); f[1] = bf16_hi(q.x); f[2] = bf16_lo(q.y); f[3] = bf16_hi(q.y);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] *= c;
    if constexpr (sizeof(O) == 4)
      *reinterpret_cast<float4*>(out + head + i * VEC) = make_float4(f[0], f[1], f[2], f[3]);
    else
      *reinterpret_cast<uint2*>(out + head + i * VEC) =
          make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  }
  const int tail = head + vecs * VEC;
  for (int i = threadIdx.x; i < head + (n - tail); i += kThreads) {
    const int e = i < head ? i : tail + (i - head);
    const float f[1] = {to_f32(in[e]) * c};
    store_vec<O, 1>(out + e, f);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
grad_clip_kernel(const __grid_constant__ List<N> l, const float* norm, float max_norm) {
  const float v = *norm;
  float c = 1.f;
  if (isfinite(v)) c = fminf(1.f, max_norm / (v + 1e-6f));
  // from the last chunk down: what the norm read last is still in L2
  for (int k = l.n_chunks - 1 - blockIdx.x; k >= 0; k -= gridDim.x) {
    const int t = tensor_of(l, k);
    if (c == 1.f && l.in[t] == l.out[t]) continue;   // in place: nothing changes
    const long long off = static_cast<long long>(k - l.first[t]) * kChunk;
    const long long left = l.numel[t] - off;
    const int n = static_cast<int>(left < kChunk ? left : kChunk);
    const __nv_bfloat16* ib = static_cast<const __nv_bfloat16*>(l.in[t]) + off;
    const float* fi = static_cast<const float*>(l.in[t]) + off;
    __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(l.out[t]) + off;
    float* fo = static_cast<float*>(l.out[t]) + off;
    switch (l.kind[t]) {
      case 0: scale_chunk(fi, fo, n, c); break;
      case 1: scale_chunk(ib, fo, n, c); break;
      case 2: scale_chunk(fi, ob, n, c); break;
      default: scale_chunk(ib, ob, n, c); break;
    }
  }
}

// Tensors [at, at + N) of the list, the empty ones left out; returns where the
// next launch goes on.
template <int N>
int fill(List<N>& l, const ClipTensor* t, int n, int at) {
  l.n = 0;
  long long chunks = 0;
  for (; at < n && l.n < N; ++at) {
    if (t[at].numel == 0) continue;
    const long long c = (t[at].numel + kChunk - 1) / kChunk;
    if (chunks + c > 0x7fffffffLL) break;
    const int i = l.n++;
    l.in[i] = t[at].in;
    l.out[i] = t[at].out;
    l.numel[i] = t[at].numel;
    l.first[i] = static_cast<int>(chunks);
    l.kind[i] = static_cast<unsigned char>((t[at].in_bf16 ? 1 : 0) | (t[at].out_bf16 ? 2 : 0));
    chunks += c;
  }
  l.n_chunks = static_cast<int>(chunks);
  return at;
}

int ctas(int chunks, int num_sms) {
  int g = num_sms * 8;
  if (g > kMaxCtas) g = kMaxCtas;
  return chunks < g ? chunks : g;
}

template <int N>
cudaError_t norm_lists(const ClipTensor* t, int n, double* partial, int* n_partial, int num_sms,
                       cudaStream_t s) {
  List<N> l;
  for (int at = 0; at < n;) {
    at = fill(l, t, n, at);
    if (l.n_chunks == 0) continue;
    const int g = ctas(l.n_chunks, num_sms);
    grad_squares_kernel<N><<<g, kThreads, 0, s>>>(l, partial + *n_partial);
    *n_partial += g;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N>
cudaError_t clip_lists(const ClipTensor* t, int n, const float* norm, float max_norm, int num_sms,
                       cudaStream_t s) {
  List<N> l;
  for (int at = 0; at < n;) {
    at = fill(l, t, n, at);
    if (l.n_chunks == 0) continue;
    grad_clip_kernel<N><<<ctas(l.n_chunks, num_sms), kThreads, 0, s>>>(l, norm, max_norm);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t clip_workspace_bytes(long long n) {
  const long long lists = n <= kSmallList ? 1 : (n + kLargeList - 1) / kLargeList;
  return static_cast<size_t>(lists) * kMaxCtas * sizeof(double);
}

cudaError_t launch_grad_norm(const ClipTensor* t, int n, double* partial, float* norm, int num_sms,
                             cudaStream_t s) {
  int np = 0;
  const cudaError_t e = n <= kSmallList
                            ? norm_lists<kSmallList>(t, n, partial, &np, num_sms, s)
                            : norm_lists<kLargeList>(t, n, partial, &np, num_sms, s);
  if (e != cudaSuccess) return e;
  grad_norm_kernel<<<1, kThreads, 0, s>>>(partial, np, norm);
  return cudaGetLastError();
}

cudaError_t launch_grad_clip(const ClipTensor* t, int n, const float* norm, float max_norm,
                             int num_sms, cudaStream_t s) {
  return n <= kSmallList ? clip_lists<kSmallList>(t, n, norm, max_norm, num_sms, s)
                         : clip_lists<kLargeList>(t, n, norm, max_norm, num_sms, s);
}

}  // namespace eas
