// Global norm of a list of gradients, and clipping.
//
//   norm = sqrt(sum over every tensor of g^2),
//   c = min(1, max_norm / (norm + 1e-6)),  out = c g   (c = 1: norm not finite).
//
// The list travels as a kernel argument: no table in device memory, no copy,
// and a captured graph holds its own.  Work is cut into chunks of equal length
// over all tensors; a CTA finds a chunk's tensor by bisection.  Squares are
// added up in fp32 over 32 elements and beyond that with their rounding errors
// kept (Squares).  Every CTA leaves one fp64 partial sum; the clipping CTAs each add the
// partials up themselves, in one order, so the norm needs no launch of its own
// and results repeat to the bit.
#include "eas_device.cuh"
#include "eas_launch.cuh"
#include "eas_ops.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxLogChunk = 14;     // elements a chunk: 2^10 .. 2^14
constexpr int kMinLogChunk = 10;
constexpr int kMaxCtas = 1216;       // partials a launch leaves at most
constexpr int kSmallList = 128;
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
  int log_chunk;
};

// The tensor that a chunk belongs to.  The last 32 candidates are compared at
// once, a lane each: a bisection to the end is a chain of first-time loads of
// the argument, 18 tensors took five of them in a row.
template <int N>
__device__ __forceinline__ int tensor_of(const List<N>& l, int chunk) {
  int lo = 0, hi = l.n;
  while (hi - lo > 32) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  const int i = lo + (threadIdx.x & 31);
  return lo + __popc(__ballot_sync(0xffffffffu, i < hi && l.first[i] <= chunk)) - 1;
}

// A running sum of squares: hi + lo in fp32, exact to about 2^-48 (each group's
// sum is added with its rounding error kept, Knuth's two-sum), and in fp64 what
// leaves the range in which that holds.  fp64 sums from each 16-byte load on
// were built first: this part's fp64 rate is far below its fp32 rate, and the
// norm and clipping of 1.33 G gradients (0.53 G fp32, 0.81 G bf16, into bf16)
// took 3370 us; this way 1476, which is the time of reading everything twice
// and writing it once (10.1 GB at 6.8 TB/s).  With the errors inside the groups
// of 32 kept as well it took 1540; without, a group of equal fp32 values, whose
// errors all point one way, is off by less than 2^-24 in the norm (at most 0.75
// 2^-24 over 2 million values), and equal bf16 values are exact.
struct Squares {
  float hi = 0.f, lo = 0.f;
  double rest = 0.0;

  __device__ __forceinline__ void add(float s) {
    const float t = hi + s;
    const float b = t - hi;
    lo += (hi - (t - b)) + (s - b);
    hi = t;
  }
  __device__ __forceinline__ double total() const {
    return static_cast<double>(hi) + static_cast<double>(lo) + rest;
  }
};

// Adds the squares of a group of elements.  Where their fp32 sum could have
// lost some (a gradient over 1e15 or everything below 1e-15) they are taken
// again in fp64; a group of zeros is not.
template <int U, int VEC>
__device__ __forceinline__ void add_squares(Squares& acc, const float (&f)[U][VEC]) {
  float part[U], m = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    part[u] = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) part[u] = fmaf(f[u][i], f[u][i], part[u]);
  }
#pragma unroll
  for (int o = U / 2; o > 0; o /= 2)
#pragma unroll
    for (int u = 0; u < o; ++u) part[u] += part[u + o];
  const float s = part[0];
  if (s > 1e-30f && s < 1e30f) {
    acc.add(s);
    return;
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(f[u][i]));
  if (s == 0.f && m == 0.f) return;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc.rest += static_cast<double>(f[u][i]) * f[u][i];
}

// Elements before the first 16-byte boundary at or after p.
template <typename T>
__device__ __forceinline__ int head_of(const T* p) {
  return static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
}

template <typename T>
__device__ __forceinline__ void chunk_squares(Squares& acc, const T* p, int n) {
  constexpr int VEC = kVec16<T>;
  constexpr int U = 32 / VEC;          // 32 elements a group
  int head = head_of(p);
  if (head > n) head = n;
  const int vecs = (n - head) / VEC;
  const T* v = p + head;
  int i = threadIdx.x;
  for (; i + (U - 1) * kThreads < vecs; i += U * kThreads) {
    Raw<T, VEC> raw[U];
    float f[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = load_raw<T, VEC>(v + static_cast<long long>(i + u * kThreads) * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u) widen<T, VEC>(raw[u], f[u]);
    add_squares<U, VEC>(acc, f);
  }
  for (; i < vecs; i += kThreads) {
    float f[1][VEC];
    widen<T, VEC>(load_raw<T, VEC>(v + static_cast<long long>(i) * VEC), f[0]);
    add_squares<1, VEC>(acc, f);
  }
  const int tail = head + vecs * VEC;
  for (i = threadIdx.x; i < head + (n - tail); i += kThreads) {
    const float f[1][1] = {{to_f32(p[i < head ? i : tail + (i - head)])}};
    add_squares<1, 1>(acc, f);
  }
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
  launch_dependents();
  Squares acc;
  for (int k = blockIdx.x; k < l.n_chunks; k += gridDim.x) {
    const int t = tensor_of(l, k);
    const long long off = static_cast<long long>(k - l.first[t]) << l.log_chunk;
    const long long left = l.numel[t] - off;
    const int n = static_cast<int>(left < (1 << l.log_chunk) ? left : (1 << l.log_chunk));
    if (l.kind[t] & 1)
      chunk_squares(acc, static_cast<const __nv_bfloat16*>(l.in[t]) + off, n);
    else
      chunk_squares(acc, static_cast<const float*>(l.in[t]) + off, n);
  }
  const double sum = block_sum(acc.total(), sm);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The sum of squares from the partial sums, the same to the bit in whatever CTA asks.
__device__ __forceinline__ double squares_of(const double* partial, int n, double* sm) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += partial[i];
  return block_sum(acc, sm);
}

__global__ void __launch_bounds__(kThreads)
grad_norm_kernel(const double* partial, int n, float* norm, DevStatus* st) {
  __shared__ double sm[kThreads / 32];
  wait_for_launch_before();
  const double sum = squares_of(partial, n, sm);
  if (threadIdx.x == 0) {
    *norm = static_cast<float>(sqrt(sum));
    *st = DevStatus{};   // nothing here can fail on the device
  }
}

template <typename I, typename O>
__device__ __forceinline__ void scale_chunk(const I* in, O* out, int n, float c) {
  constexpr int VEC = kVec16<I>;       // 16 bytes of input
  constexpr int W = kVec16<O> < VEC ? kVec16<O> : VEC;
  constexpr int U = 4;
  int head = head_of(in);
  if (head > n) head = n;
  // a vector's output is 16 bytes or two halves of them
  const bool vec = (reinterpret_cast<uintptr_t>(out + head) % (W * sizeof(O))) == 0;
  const int vecs = vec ? (n - head) / VEC : 0;
  for (int i0 = threadIdx.x; i0 < vecs; i0 += U * kThreads) {
    Raw<I, VEC> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kThreads < vecs)
        raw[u] = load_raw<I, VEC>(in + head + static_cast<long long>(i0 + u * kThreads) * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * kThreads >= vecs) break;
      O* to = out + head + static_cast<long long>(i0 + u * kThreads) * VEC;
      float f[VEC];
      widen<I, VEC>(raw[u], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] *= c;
      if constexpr (sizeof(O) == sizeof(I)) {
        store_vec<O, VEC>(to, f);
      } else if constexpr (sizeof(O) == 4) {
        *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
      } else {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
      }
    }
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
grad_clip_kernel(const __grid_constant__ List<N> l, const double* partial, int n_partial,
                 float* norm, float max_norm, DevStatus* st) {
  __shared__ double sm[kThreads / 32];
  __shared__ float factor;
  // the first chunk's tensor is looked up while the norm is on its way
  int k = l.n_chunks - 1 - blockIdx.x;
  int t = tensor_of(l, k);
  wait_for_launch_before();
  const double sum = squares_of(partial, n_partial, sm);
  if (threadIdx.x == 0) {
    // norm and factor in 64 bits, each rounded once: an error in the factor would
    // be every gradient's
    const double v = sqrt(sum);
    const float rounded = static_cast<float>(v);
    factor = isfinite(rounded) ? static_cast<float>(fmin(1.0, max_norm / (v + 1e-6))) : 1.f;
    if (blockIdx.x == 0) {
      *norm = rounded;
      *st = DevStatus{};
    }
  }
  __syncthreads();
  const float c = factor;
  // from the last chunk down: what the norm read last is still in L2
  for (; k >= 0; k -= gridDim.x, t = k >= 0 ? tensor_of(l, k) : 0) {
    if (c == 1.f && l.in[t] == l.out[t]) continue;   // in place: nothing changes
    const long long off = static_cast<long long>(k - l.first[t]) << l.log_chunk;
    const long long left = l.numel[t] - off;
    const int n = static_cast<int>(left < (1 << l.log_chunk) ? left : (1 << l.log_chunk));
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

// log2 of the chunk: the largest that still gives every resident CTA one, so
// that a short list is spread over the machine and a long one searches less.
int log_chunk_of(const ClipTensor* t, int n, int num_sms) {
  long long total = 0;
  for (int i = 0; i < n; ++i) total += t[i].numel;
  int lc = kMaxLogChunk;
  while (lc > kMinLogChunk && (total >> lc) < 8LL * num_sms) --lc;
  return lc;
}

// Tensors [at, at + N) of the list, the empty ones left out; returns where the
// next launch goes on.
template <int N>
int fill(List<N>& l, const ClipTensor* t, int n, int at, int log_chunk) {
  l.n = 0;
  l.log_chunk = log_chunk;
  long long chunks = 0;
  for (; at < n && l.n < N; ++at) {
    if (t[at].numel == 0) continue;
    const long long c = (t[at].numel + (1LL << log_chunk) - 1) >> log_chunk;
    if (chunks + c > 0x7fffffffLL) break;   // never the first: numel <= 2^40
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
cudaError_t launch_lists(const ClipTensor* t, int n, bool clip, float max_norm, double* partial,
                         float* norm, DevStatus* st, int num_sms, cudaStream_t s) {
  const int lc = log_chunk_of(t, n, num_sms);
  List<N> l;
  int np = 0;
  for (int at = 0; at < n;) {
    at = fill(l, t, n, at, lc);
    if (l.n_chunks == 0) continue;
    const int g = ctas(l.n_chunks, num_sms);
    grad_squares_kernel<N><<<g, kThreads, 0, s>>>(l, partial + np);
    np += g;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (!clip || np == 0)
    return launch_overlapped(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, partial, np, norm,
                             st);
  for (int at = 0; at < n;) {
    at = fill(l, t, n, at, lc);
    if (l.n_chunks == 0) continue;
    e = launch_overlapped(grad_clip_kernel<N>, dim3(ctas(l.n_chunks, num_sms)), dim3(kThreads), 0, s,
                          l, partial, np, norm, max_norm, st);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace

size_t clip_workspace_bytes(long long n) {
  const long long lists = n <= kSmallList ? 1 : (n + kLargeList - 1) / kLargeList;
  return static_cast<size_t>(lists) * kMaxCtas * sizeof(double);
}

cudaError_t launch_clip_grad_norm(const ClipTensor* t, int n, bool clip, float max_norm,
                                  double* partial, float* norm, DevStatus* st, int num_sms,
                                  cudaStream_t s) {
  return n <= kSmallList
             ? launch_lists<kSmallList>(t, n, clip, max_norm, partial, norm, st, num_sms, s)
             : launch_lists<kLargeList>(t, n, clip, max_norm, partial, norm, st, num_sms, s);
}

}  // namespace eas
