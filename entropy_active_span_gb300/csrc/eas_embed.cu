// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale E[id_t] (zero for padding),
//   dE[v]  = scale * sum over the tokens t with id_t = v of dout[t].
//
// The gradient sorts the tokens by id (stable radix sort, so the tokens of a
// row stay in their order), cuts the sorted list into chunks of equal length
// and sums each chunk's runs of equal ids in fp32 registers.  A run that lies
// in one chunk is written to its row of dE at once; the pieces of a run that
// crosses chunks go to scratch and are added in order by a second kernel.  No
// floating-point atomics: results repeat to the bit.
#include "eas_device.cuh"
#include "eas_kernels.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr int kWhereEmbed = 20;

// ------------------------------------------------------------------ lookup

// CTA (x, y): rows x * blockDim.y + threadIdx.y.  CTA 0 also checks every id
// and writes the status word: no other launch clears it.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
embed_fwd_kernel(const EmbedFwdArgs p) {
  if (p.status && blockIdx.x == 0) {
    __shared__ unsigned long long first_bad;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    if (tid == 0) first_bad = ~0ull;
    __syncthreads();
    for (long long t = tid; t < p.T; t += 256) {
      const int id = p.ids[t];
      if (id < -1 || id >= p.V) {
        atomicMin(&first_bad, static_cast<unsigned long long>(t));
        break;
      }
    }
    __syncthreads();
    if (tid == 0) {
      const bool bad = first_bad != ~0ull;
      p.status->code = bad ? kStInvalidArg : kStOk;
      p.status->where = bad ? kWhereEmbed : 0;
      p.status->info = bad ? static_cast<int>(first_bad) : 0;
    }
  }
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= p.T) return;
  const int id = p.ids[t];
  const bool real = id >= 0 && id < p.V;
  const T* src = static_cast<const T*>(p.table) + static_cast<long long>(real ? id : 0) * p.H;
  T* dst = static_cast<T*>(p.out) + t * p.H;
#pragma unroll 4
  for (int c = threadIdx.x * VEC; c < p.H; c += blockDim.x * VEC) {
    float f[VEC] = {};
    if (real) {
      widen<T, VEC>(load_raw<T, VEC>(src + c), f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] *= p.scale;
    }
    store_vec<T, VEC>(dst + c, f);
  }
}

// -------------------------------------------------------------------- sort

// LSD radix sort of (id, token), kSortBins digits a pass.  A tile is a
// multiple of kSortSub tokens so that there are at most kSortTiles tiles.
constexpr int kSortBits = 9;
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortThreads = 512;            // one a digit in the offset step
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 4;
constexpr int kSortSub = kSortThreads * kSortRounds;
constexpr int kSortTiles = 128;

struct SortPass {
  const int* ids;         // first pass: the token ids; later: null
  const int* keys_in;
  const int* pos_in;
  int* keys_out;
  int* pos_out;
  int* hist;              // [n_tiles][kSortBins]
  long long T;
  int V;
  int shift;
  int n_tiles;
  long long tile;         // tokens a tile
  DevStatus* status;
};

__device__ __forceinline__ int sort_key(const SortPass& p, long long i) {
  if (!p.ids) return p.keys_in[i];
  const int id = p.ids[i];
  return id >= 0 && id < p.V ? id : p.V;     // padding and bad ids go last
}

__global__ void __launch_bounds__(kSortThreads) sort_hist_kernel(const SortPass p) {
  __shared__ int cnt[kSortBins];
  cnt[threadIdx.x] = 0;
  __syncthreads();
  const long long lo = blockIdx.x * p.tile;
  const long long hi = lo + p.tile < p.T ? lo + p.tile : p.T;
  for (long long i = lo + threadIdx.x; i < hi; i += kSortThreads) {
    if (p.ids) {
      const int id = p.ids[i];
      if (id < -1 || id >= p.V) report(p.status, kStInvalidArg, kWhereEmbed, static_cast<int>(i));
    }
    atomicAdd(&cnt[(sort_key(p, i) >> p.shift) & (kSortBins - 1)], 1);
  }
  __syncthreads();
  p.hist[blockIdx.x * kSortBins + threadIdx.x] = cnt[threadIdx.x];
}

// Stable: a warp takes 32 * kSortRounds consecutive tokens, ranks them among
// its own, and the warps' counts are added up in order.
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const SortPass p) {
  __shared__ int cnt[kSortWarps][kSortBins];
  __shared__ int warp_sum[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // where this tile's tokens of digit `tid` start
  int before = 0, total = 0;
  for (int t = 0; t < p.n_tiles; ++t) {
    const int n = p.hist[t * kSortBins + tid];
    if (t < blockIdx.x) before += n;
    total += n;
  }
  int x = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int base = before + x - total;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];

  const long long lo = blockIdx.x * p.tile;
  const long long hi = lo + p.tile < p.T ? lo + p.tile : p.T;
  for (long long sub = lo; sub < hi; sub += kSortSub) {
    for (int w = 0; w < kSortWarps; ++w) cnt[w][tid] = 0;
    __syncthreads();
    int key[kSortRounds], pos[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      const long long i = sub + warp * (32 * kSortRounds) + r * 32 + lane;
      const bool in = i < hi;
      key[r] = in ? sort_key(p, i) : -1;
      pos[r] = in ? (p.ids ? static_cast<int>(i) : p.pos_in[i]) : 0;
      const int digit = in ? (key[r] >> p.shift) & (kSortBins - 1) : kSortBins;
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      const int mine = __popc(same & ((1u << lane) - 1));
      rank[r] = mine;
      if (in) rank[r] += cnt[warp][digit];
      __syncwarp();
      if (in && mine == 0) cnt[warp][digit] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    int at = base;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = cnt[w][tid];
      cnt[w][tid] = at;
      at += n;
    }
    base = at;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      if (key[r] >= 0) {
        const int to = cnt[warp][(key[r] >> p.shift) & (kSortBins - 1)] + rank[r];
        p.keys_out[to] = key[r];
        p.pos_out[to] = pos[r];
      }
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------- summation

struct SumArgs {
  const int* keys;        // sorted ids; V: padding
  const int* pos;         // their tokens
  const void* dout;
  float* dw;
  float* partial;         // [n_chunks][2][H]: piece of a run from before, piece of a run that goes on
  long long T;
  int V, H;
  int chunk;
  float scale;
  int accumulate;
};

template <int VEC>
__device__ __forceinline__ void put_row(float* dst, const float (&acc)[VEC], float scale, int add) {
  float o[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = acc[i] * scale;
  constexpr int W = VEC == 1 ? 1 : 4;
#pragma unroll
  for (int h = 0; h < VEC; h += W) {
    float v[W];
    if (add) widen<float, W>(load_raw<float, W>(dst + h), v);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = add ? v[i] + o[h + i] : o[h + i];
    store_vec<float, W>(dst + h, v);
  }
}

constexpr int kSumThreads = 128;
constexpr int kSumUnroll = 8;
constexpr int kMaxChunk = 128;

// CTA (x, y): chunk x of the sorted tokens, kSumThreads * VEC columns.
template <typename T, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumArgs p) {
  __shared__ int keys[kMaxChunk + 2];   // [0]: the key before the chunk, [n + 1]: the one after
  __shared__ int pos[kMaxChunk];
  const long long i0 = static_cast<long long>(blockIdx.x) * p.chunk;
  const int n = static_cast<int>(p.T - i0 < p.chunk ? p.T - i0 : p.chunk);
  for (int i = threadIdx.x; i < n + 2; i += kSumThreads) {
    const long long k = i0 + i - 1;
    keys[i] = k >= 0 && k < p.T ? p.keys[k] : -1;
    if (i < n) pos[i] = p.pos[i0 + i];
  }
  __syncthreads();
  const int c = (blockIdx.y * kSumThreads + threadIdx.x) * VEC;
  if (c >= p.H) return;
  const T* dout = static_cast<const T*>(p.dout) + c;
  float acc[VEC] = {};
  int start = 0;                        // where the current run starts in the chunk
  for (int i = 0; i < n; i += kSumUnroll) {
    if (keys[i + 1] == p.V) break;      // the padding, after every token
    Raw<T, VEC> raw[kSumUnroll];
#pragma unroll
    for (int u = 0; u < kSumUnroll; ++u)
      if (i + u < n && keys[i + u + 1] != p.V)
        raw[u] = load_raw<T, VEC>(dout + static_cast<long long>(pos[i + u]) * p.H);
#pragma unroll
    for (int u = 0; u < kSumUnroll; ++u) {
      const int k = i + u;
      if (k < n && keys[k + 1] != p.V) {
        float f[VEC];
        widen<T, VEC>(raw[u], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += f[e];
        const int key = keys[k + 1];
        if (k + 1 == n || keys[k + 2] != key) {   // the run ends here, or the chunk does
          const bool from_before = start == 0 && keys[0] == key;
          const bool goes_on = keys[k + 2] == key;
          if (!from_before && !goes_on) {
            put_row<VEC>(p.dw + static_cast<long long>(key) * p.H + c, acc, p.scale, p.accumulate);
          } else {
            float* q = p.partial + (2ll * blockIdx.x + (from_before ? 0 : 1)) * p.H + c;
            put_row<VEC>(q, acc, 1.f, 0);
          }
          start = k + 1;
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
        }
      }
    }
  }
}

// Adds up the runs that cross chunks: the CTAs of the chunk in which a run
// starts walk the chunks it covers.
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const SumArgs p, int n_chunks) {
  const long long end = static_cast<long long>(blockIdx.x + 1) * p.chunk;
  if (end >= p.T) return;
  const int key = p.keys[end - 1];
  if (key == p.V || p.keys[end] != key) return;                      // no run goes on
  const long long begin = end - p.chunk;
  if (p.keys[begin] == key && begin > 0 && p.keys[begin - 1] == key) return;   // nor starts here
  // the last chunk of the run: the last that begins with its id
  int last = blockIdx.x + 1, hi = n_chunks;
  while (hi - last > 1) {
    const int mid = last + (hi - last) / 2;
    if (p.keys[static_cast<long long>(mid) * p.chunk] == key) last = mid; else hi = mid;
  }
  const int c = blockIdx.y * kSumThreads + threadIdx.x;
  if (c >= p.H) return;
  float acc = p.partial[(2ll * blockIdx.x + 1) * p.H + c];
#pragma unroll 8
  for (int k = blockIdx.x + 1; k <= last; ++k) acc += p.partial[2ll * k * p.H + c];
  const float a[1] = {acc};
  put_row<1>(p.dw + static_cast<long long>(key) * p.H + c, a, p.scale, p.accumulate);
}

// Zeros in the rows of dw that no token touches: a row's id is looked up in
// the sorted list.
constexpr int kZeroRows = 8;
template <int VEC>
__global__ void __launch_bounds__(256) embed_zero_kernel(const SumArgs p) {
  __shared__ int skip[kZeroRows];
  const int v0 = blockIdx.x * kZeroRows;
  if (threadIdx.x < kZeroRows) {
    const int v = v0 + threadIdx.x;
    long long lo = 0, hi = p.T;
    while (lo < hi) {
      const long long mid = (lo + hi) >> 1;
      if (p.keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    skip[threadIdx.x] = v >= p.V || (lo < p.T && p.keys[lo] == v);
  }
  __syncthreads();
  const float z[VEC] = {};
  for (int r = 0; r < kZeroRows; ++r) {
    if (skip[r]) continue;
    float* row = p.dw + static_cast<long long>(v0 + r) * p.H;
    for (int c = threadIdx.x * VEC; c < p.H; c += 256 * VEC) store_vec<float, VEC>(row + c, z);
  }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

long long sort_tile(long long T) {
  const long long most = static_cast<long long>(kSortTiles) * kSortSub;
  return kSortSub * (T > most ? (T + most - 1) / most : 1);
}

SumArgs sum_args(const EmbedBwdArgs& a, const EmbedBwdPlan& pl, int buf) {
  SumArgs s;
  s.keys = reinterpret_cast<const int*>(a.scratch + pl.keys[buf]);
  s.pos = reinterpret_cast<const int*>(a.scratch + pl.pos[buf]);
  s.dout = a.dout;
  s.dw = a.dw;
  s.partial = reinterpret_cast<float*>(a.scratch + pl.partial);
  s.T = a.T;
  s.V = a.V;
  s.H = a.H;
  s.chunk = pl.chunk;
  s.scale = a.scale;
  s.accumulate = a.accumulate;
  return s;
}

int sort_passes(int V) {
  int bits = 1;
  while (bits < 31 && (V >> bits) != 0) ++bits;   // keys 0 .. V
  return (bits + kSortBits - 1) / kSortBits;
}

}  // namespace

cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, int is_bf16, cudaStream_t s) {
  const int vec16 = is_bf16 ? 8 : 4;
  const int vec = a.H % vec16 == 0 ? vec16 : 1;
  int tx = 32;
  while (tx < 256 && tx * vec < a.H) tx *= 2;
  const dim3 block(tx, 256 / tx);
  const long long grid = a.T > 0 ? (a.T + block.y - 1) / block.y : 1;
  const unsigned g = static_cast<unsigned>(grid);
  if (is_bf16) {
    if (vec == 1) embed_fwd_kernel<__nv_bfloat16, 1><<<g, block, 0, s>>>(a);
    else embed_fwd_kernel<__nv_bfloat16, 8><<<g, block, 0, s>>>(a);
  } else {
    if (vec == 1) embed_fwd_kernel<float, 1><<<g, block, 0, s>>>(a);
    else embed_fwd_kernel<float, 4><<<g, block, 0, s>>>(a);
  }
  return cudaGetLastError();
}

// A worker's chunk is as long as 4096 workers allow (a worker is a chunk and
// 512 columns), 16 to 128 tokens: short chunks keep small calls parallel, long
// ones keep the pieces of runs few.
EmbedBwdPlan embed_bwd_plan(long long T, long long H, long long V) {
  (void)V;
  EmbedBwdPlan p;
  const long long cols = (H + 511) / 512;
  p.chunk = kMaxChunk;
  while (p.chunk > 16 && (T + p.chunk - 1) / p.chunk * cols < 4096) p.chunk /= 2;
  const size_t n = static_cast<size_t>(T > 0 ? T : 1);
  size_t o = 0;
  for (int b = 0; b < 2; ++b) {
    p.keys[b] = o; o = up(o + 4 * n);
    p.pos[b] = o; o = up(o + 4 * n);
  }
  p.hist = o; o = up(o + sizeof(int) * kSortTiles * kSortBins);
  p.partial = o;
  const size_t chunks = (n + p.chunk - 1) / p.chunk;
  if (chunks > 1) o = up(o + chunks * 2 * 4 * static_cast<size_t>(H));
  p.total = o;
  return p;
}

cudaError_t launch_embed_sort(const EmbedBwdArgs& a, cudaStream_t s) {
  const EmbedBwdPlan pl = embed_bwd_plan(a.T, a.H, a.V);
  const int passes = sort_passes(a.V);
  for (int i = 0; i < passes; ++i) {
    SortPass p;
    p.ids = i == 0 ? a.ids : nullptr;
    p.keys_in = reinterpret_cast<const int*>(a.scratch + pl.keys[(i + 1) & 1]);
    p.pos_in = reinterpret_cast<const int*>(a.scratch + pl.pos[(i + 1) & 1]);
    p.keys_out = reinterpret_cast<int*>(a.scratch + pl.keys[i & 1]);
    p.pos_out = reinterpret_cast<int*>(a.scratch + pl.pos[i & 1]);
    p.hist = reinterpret_cast<int*>(a.scratch + pl.hist);
    p.T = a.T;
    p.V = a.V;
    p.shift = i * kSortBits;
    p.tile = sort_tile(a.T);
    p.n_tiles = static_cast<int>((a.T + p.tile - 1) / p.tile);
    p.status = a.status;
    sort_hist_kernel<<<p.n_tiles, kSortThreads, 0, s>>>(p);
    sort_scatter_kernel<<<p.n_tiles, kSortThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int VEC>
static void sum_t(const SumArgs& s, int n_chunks, cudaStream_t st) {
  const dim3 grid(n_chunks, (s.H + kSumThreads * VEC - 1) / (kSumThreads * VEC));
  embed_sum_kernel<T, VEC><<<grid, kSumThreads, 0, st>>>(s);
}

cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, int is_bf16, cudaStream_t st) {
  const EmbedBwdPlan pl = embed_bwd_plan(a.T, a.H, a.V);
  const SumArgs s = sum_args(a, pl, (sort_passes(a.V) - 1) & 1);
  if (!a.accumulate) {
    const unsigned g = static_cast<unsigned>((static_cast<long long>(a.V) + kZeroRows - 1) / kZeroRows);
    if (a.H % 4 == 0) embed_zero_kernel<4><<<g, 256, 0, st>>>(s);
    else embed_zero_kernel<1><<<g, 256, 0, st>>>(s);
  }
  if (a.T == 0) return cudaGetLastError();
  const int n_chunks = static_cast<int>((a.T + pl.chunk - 1) / pl.chunk);
  const int vec16 = is_bf16 ? 8 : 4;
  if (a.H % vec16 == 0) {
    if (is_bf16) sum_t<__nv_bfloat16, 8>(s, n_chunks, st);
    else sum_t<float, 4>(s, n_chunks, st);
  } else {
    if (is_bf16) sum_t<__nv_bfloat16, 1>(s, n_chunks, st);
    else sum_t<float, 1>(s, n_chunks, st);
  }
  if (n_chunks > 1)
    embed_join_kernel<<<dim3(n_chunks, (a.H + kSumThreads - 1) / kSumThreads), kSumThreads, 0, st>>>(s, n_chunks);
  return cudaGetLastError();
}

}  // namespace eas
