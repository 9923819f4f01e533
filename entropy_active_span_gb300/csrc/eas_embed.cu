// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale E[id_t] (zero for padding),
//   dE[v]  = scale * sum over the tokens t with id_t = v of dout[t].
//
// The gradient sorts the tokens by id (stable radix sort, so the tokens of a
// row stay in their order), cuts the sorted list into chunks of equal length
// and sums each chunk's runs of equal ids in fp32 registers.  A run that lies
// in two chunks at most is written to its row of dE at once; the pieces of a
// longer one go to scratch and are added in order by a second kernel.  Lists of
// up to 512 tokens need no sort.  No floating-point atomics: results repeat to
// the bit.
//
// All of it is bound by bytes: dout is read once, dE written once.  16384 tokens
// into [128256, 4096] take 329 us and 131072 Zipf-distributed ones into [129280,
// 7168] 785 us, both 6.8 TB/s; the plain copy rate is 6.8.
#include "eas_device.cuh"
#include "eas_launch.cuh"
#include "eas_ops.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr int kWhereEmbed = 20;

// ------------------------------------------------------------------ lookup

// Vectors of a row that a thread holds at a time: single elements (rows of odd
// width) go four together, so that as many loads are on their way.
template <int VEC>
constexpr int kCols = VEC == 1 ? 4 : 1;

template <typename T, int VEC, int kRows>
__global__ void __launch_bounds__(256)
embed_fwd_kernel(const EmbedFwdArgs p) {
  // kRows rows a thread: their ids come in one latency and their loads leave
  // together
  const long long t0 = (static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y) * kRows;
  const T* src[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int id = t0 + r < p.T ? p.ids[t0 + r] : -1;
    src[r] = id >= 0 && id < p.V ? static_cast<const T*>(p.table) + static_cast<long long>(id) * p.H : nullptr;
    if (p.status && id != -1 && !src[r] && threadIdx.x == 0)
      report(p.status, kStInvalidArg, kWhereEmbed, static_cast<int>(t0 + r));
  }
  T* dst = static_cast<T*>(p.out) + t0 * p.H;
  const int step = blockDim.x * VEC;
  for (int c0 = threadIdx.x * VEC; c0 < p.H; c0 += kCols<VEC> * step) {
    Raw<T, VEC> raw[kCols<VEC>][kRows];
#pragma unroll
    for (int m = 0; m < kCols<VEC>; ++m)
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (src[r] && c0 + m * step < p.H) raw[m][r] = load_const<T, VEC>(src[r] + c0 + m * step);
#pragma unroll
    for (int m = 0; m < kCols<VEC>; ++m) {
      const int c = c0 + m * step;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (t0 + r >= p.T || c >= p.H) break;
        float f[VEC] = {};
        if (src[r]) {
          widen<T, VEC>(raw[m][r], f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) f[i] *= p.scale;
        }
        // the table's rows come again, the output does not: 130 us against 134 at
        // [65536, 5120] bf16 with Zipf-distributed ids
        store_vec<T, VEC, true>(dst + static_cast<long long>(r) * p.H + c, f);
      }
    }
  }
}

// -------------------------------------------------------------------- sort

// LSD radix sort of (id, token), kSortBins digits a pass: here over several
// launches, for lists that the cluster sort below does not hold.  A tile is a
// multiple of kSortSub tokens so that there are at most kSortTiles tiles.
constexpr int kSortBits = 9;
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortThreads = 512;            // one a digit in the offset step
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 4;
constexpr int kSortSub = kSortThreads * kSortRounds;
constexpr int kSortTiles = 128;

// The number of runs that cross chunks stands behind the status word; the sort
// clears both.
constexpr size_t kClearBytes = sizeof(DevStatus) + sizeof(int);
__host__ __device__ __forceinline__ int* run_count(DevStatus* st) { return reinterpret_cast<int*>(st + 1); }

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
  wait_for_launch_before();
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
  wait_for_launch_before();

  // where this tile's tokens of digit `tid` start
  int before = 0, total = 0;
#pragma unroll 32
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

// The whole sort in one launch, for lists that fit the shared memory of a
// cluster of eight CTAs.  CTA 0 .. 7 hold the list, 1024 * kRounds pairs each;
// a pass ranks every warp's run of digits, adds the counts up over warps and
// (through distributed shared memory) over CTAs, and moves each pair to its
// place in whichever CTA holds that.  A thread keeps its pairs in registers
// meanwhile, so one buffer is enough.  A call with 16384 tokens of 64 columns
// takes 28 us this way; at 131072 tokens the eight CTAs sorted for 75 us against
// 33 of the launches above, which is why the lists end at 32768.
constexpr int kClusterCtas = 8;
constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterThreads / 32;
constexpr int kClusterRounds = 4;
constexpr long long kClusterMost = 1ll * kClusterCtas * kClusterThreads * kClusterRounds;

struct ClusterSort {
  const int* ids;
  int* keys_out;
  int* pos_out;
  long long T;
  int V;
  int passes;
  DevStatus* status;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ int peer_load(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void peer_store2(uint32_t addr, int a, int b) {
  asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

template <int kRounds>
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kClusterThreads)
cluster_sort_kernel(const ClusterSort p) {
  constexpr int kTile = kClusterThreads * kRounds;
  // (key, token) pairs of this CTA [kTile], then counts [warps][digits]
  extern __shared__ __align__(128) unsigned char smem[];
  int2* pair = reinterpret_cast<int2*>(smem);
  unsigned short(*cnt)[kSortBins] = reinterpret_cast<unsigned short(*)[kSortBins]>(smem + sizeof(int2) * kTile);
  __shared__ int hist[kSortBins];
  __shared__ int base[kSortBins];
  __shared__ int warp_sum[kSortBins / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x;          // the first cluster: its rank is the block index
  const int T = static_cast<int>(p.T);
  if (rank == 0 && tid == 0) {
    p.status->code = kStOk;
    p.status->where = p.status->info = 0;
    *run_count(p.status) = 0;
  }
  cluster_sync();                       // the status is clear, and every CTA runs
  int key[kRounds], pos[kRounds];
  unsigned short below[kRounds];
  const int first = rank * kTile + warp * (32 * kRounds) + lane;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int i = first + 32 * r;
    key[r] = -1;
    pos[r] = i;
    if (i < T) {
      const int id = p.ids[i];
      if (id < -1 || id >= p.V) report(p.status, kStInvalidArg, kWhereEmbed, i);
      key[r] = id >= 0 && id < p.V ? id : p.V;      // padding and bad ids go last
    }
  }
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * kSortBits;
    if (pass > 0) {
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int i = first + 32 * r;
        const int2 kp = pair[i - rank * kTile];
        key[r] = i < T ? kp.x : -1;
        pos[r] = kp.y;
      }
    }
    for (int i = tid; i < kClusterWarps * kSortBins / 2; i += kClusterThreads)
      reinterpret_cast<uint32_t*>(&cnt[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int digit = key[r] >= 0 ? (key[r] >> shift) & (kSortBins - 1) : kSortBins;
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      const int mine = __popc(same & ((1u << lane) - 1));
      below[r] = static_cast<unsigned short>(mine);
      if (key[r] >= 0) below[r] += cnt[warp][digit];
      __syncwarp();
      if (key[r] >= 0 && mine == 0) cnt[warp][digit] += static_cast<unsigned short>(__popc(same));
      __syncwarp();
    }
    __syncthreads();
    if (tid < kSortBins) {
      int n = 0;
#pragma unroll 8
      for (int w = 0; w < kClusterWarps; ++w) {
        const int c = cnt[w][tid];
        cnt[w][tid] = static_cast<unsigned short>(n);
        n += c;
      }
      hist[tid] = n;
    }
    cluster_sync();                     // every CTA's counts are out, its pairs in registers
    int before = 0, total = 0, x = 0;
    if (tid < kSortBins) {
#pragma unroll
      for (int c = 0; c < kClusterCtas; ++c) {
        const int n = peer_load(peer_smem(smem_u32(&hist[tid]), c));
        if (c < rank) before += n;
        total += n;
      }
      x = total;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
    }
    __syncthreads();
    if (tid < kSortBins) {
      int at = before + x - total;
      for (int w = 0; w < warp; ++w) at += warp_sum[w];
      base[tid] = at;
    }
    __syncthreads();
    const bool last = pass + 1 == p.passes;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      if (key[r] < 0) continue;
      const int digit = (key[r] >> shift) & (kSortBins - 1);
      const int to = base[digit] + cnt[warp][digit] + below[r];
      if (last) {
        p.keys_out[to] = key[r];
        p.pos_out[to] = pos[r];
      } else {
        peer_store2(peer_smem(smem_u32(&pair[to % kTile]), to / kTile), key[r], pos[r]);
      }
    }
    cluster_sync();                     // the pairs have arrived, and hist has been read
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
  int sum_ctas;
  int zero_rows;          // rows of dw a zeroing CTA looks after
  int* n_runs;            // runs that cross chunks: how many,
  int* runs;              // and the chunk in which each starts
  int n_chunks;
};

template <int VEC>
__device__ __forceinline__ void put_row(float* dst, const float (&acc)[VEC], float scale, int add) {
  float o[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) o[i] = acc[i] * scale;
  constexpr int W = VEC < 4 ? 1 : 4;
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
template <int VEC>
constexpr int kSumUnroll = VEC == 1 ? 4 : 8;   // tokens on their way
constexpr int kMaxChunk = 128;

// Zeros in the n floats at p by a warp; p need not start on a 16-byte boundary
// (rows of odd width).
__device__ __forceinline__ void zero_floats(float* p, int n, int lane) {
  int head = static_cast<int>(-(reinterpret_cast<uintptr_t>(p) >> 2) & 3);
  if (head > n) head = n;
  const int mid = (n - head) & ~3;
#pragma unroll 4
  for (int c = lane * 4; c < mid; c += 128)
    *reinterpret_cast<float4*>(p + head + c) = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < n - mid) p[lane < head ? lane : mid + lane] = 0.f;
}

// Zeros in those of the CTA's rows of dw (from v0) whose skip[] is 0, a warp a row.
__device__ __forceinline__ void zero_rows(const SumArgs& p, long long v0, const int* skip, int tid) {
#pragma unroll 2
  for (int r = tid >> 5; r < p.zero_rows; r += kSumThreads / 32)
    if (!skip[r]) zero_floats(p.dw + (v0 + r) * p.H, p.H, tid & 31);
}

// The rows that no token names, for one CTA: each row's id is looked up in the
// sorted list.
__device__ __forceinline__ void zero_unnamed(const SumArgs& p, int block, int* skip) {
  const long long v0 = static_cast<long long>(block) * p.zero_rows;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  if (tid < p.zero_rows) {
    const long long v = v0 + tid;
    long long lo = 0, hi = p.T;
    while (lo < hi) {
      const long long mid = (lo + hi) >> 1;
      if (p.keys[mid] < v) lo = mid + 1; else hi = mid;
    }
    skip[tid] = v >= p.V || (lo < p.T && p.keys[lo] == v);
  }
  __syncthreads();
  zero_rows(p, v0, skip, tid);
}

// The first index from `from` on whose key is not `key`, at most `limit`; a warp.
__device__ __forceinline__ int run_end(const int* keys, int from, int limit, int key) {
  const int lane = threadIdx.x & 31;
  for (int i = from; i < limit; i += 32) {
    const unsigned m = __ballot_sync(0xffffffffu, i + lane < limit && keys[i + lane] == key);
    if (m != 0xffffffffu) return i + __popc(m);
  }
  return limit;
}

// CTA b < p.sum_ctas: blockDim.y chunks of the sorted tokens (one where the
// columns fill the CTA), blockDim.x * VEC columns of them.  The CTAs after them fill the rows that no token names, so that
// their stores run beside the others' loads.
template <typename T, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumArgs p) {
  __shared__ int key_store[4][2 * kMaxChunk + 2];
  __shared__ int pos_store[4][2 * kMaxChunk];
  wait_for_launch_before();
  if (blockIdx.x >= p.sum_ctas) {
    zero_unnamed(p, blockIdx.x - p.sum_ctas, key_store[0]);
    return;
  }
  int* keys = key_store[threadIdx.y];   // [0]: the key before the chunk; then two chunks and one more
  int* pos = pos_store[threadIdx.y];
  const int step = blockDim.x * VEC, width = kCols<VEC> * step;
  const int slabs = (p.H + width - 1) / width;
  const int group = blockIdx.x / slabs, slab = blockIdx.x - group * slabs;
  const int chunk = group * blockDim.y + threadIdx.y;
  const long long i0 = static_cast<long long>(chunk) * p.chunk;
  const long long left = p.T - i0;
  const int n = static_cast<int>(left < 0 ? 0 : left < p.chunk ? left : p.chunk);
  const int seen = static_cast<int>(left < 0 ? 0 : left < 2 * p.chunk ? left : 2 * p.chunk);
  for (int i = threadIdx.x; i < 2 * p.chunk + 2; i += blockDim.x) {
    const long long k = i0 + i - 1;
    keys[i] = k >= 0 && k < p.T ? p.keys[k] : -1;
    if (i < seen) pos[i] = p.pos[i0 + i];
  }
  // A run of at most two chunks is the work of the chunk in which it starts: it
  // goes on into the next one (to `stop`), which leaves those tokens out (to
  // `begin`).
  const bool came = n > 0 && i0 > 0 && p.keys[i0 - 1] == p.keys[i0];
  const bool came_far = came && i0 > p.chunk && p.keys[i0 - p.chunk - 1] == p.keys[i0];
  __syncthreads();
  int begin = 0, stop = n;
  const bool through = came && keys[n + 1] == keys[1];       // and goes on past the chunk
  if (came && !came_far && !through) begin = run_end(keys + 1, 0, n, keys[1]);
  if (n == p.chunk && keys[n + 1] == keys[n] && !through && keys[2 * p.chunk + 1] != keys[n])
    stop = run_end(keys + 1, n, seen, keys[n]);
  const int c = slab * width + threadIdx.x * VEC;
  if (c >= p.H) return;
  const T* dout = static_cast<const T*>(p.dout) + c;
  constexpr int U = kSumUnroll<VEC>, M = kCols<VEC>;
  float acc[M][VEC] = {};
  bool piece = came && begin == 0;      // the current run started in an earlier chunk
  for (int i = begin; i < stop; i += U) {
    if (keys[i + 1] == p.V) break;      // the padding, after every token
    Raw<T, VEC> raw[U][M];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < M; ++m)
        if (i + u < stop && keys[i + u + 1] != p.V && c + m * step < p.H)
          raw[u][m] = load_const<T, VEC>(dout + static_cast<long long>(pos[i + u]) * p.H + m * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = i + u;
      if (k < stop && keys[k + 1] != p.V) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
          float f[VEC];
          widen<T, VEC>(raw[u][m], f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[m][e] += f[e];
        }
        const int key = keys[k + 1];
        const bool goes_on = keys[k + 2] == key;
        if (!goes_on || k + 1 == stop) {          // the run ends here, or the chunk does
          const bool done = !piece && !goes_on;
          if (goes_on && !piece && threadIdx.x == 0 && slab == 0)
            p.runs[atomicAdd(p.n_runs, 1)] = chunk;
          float* to = done ? p.dw + static_cast<long long>(key) * p.H + c
                           : p.partial + (2ll * chunk + (piece ? 0 : 1)) * p.H + c;
#pragma unroll
          for (int m = 0; m < M; ++m) {
            if (c + m * step < p.H) put_row<VEC>(to + m * step, acc[m], done ? p.scale : 1.f, done && p.accumulate);
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[m][e] = 0.f;
          }
          piece = false;
        }
      }
    }
  }
}

// Adds up the runs of three chunks or more.  The sums have listed them (in any order:
// each is added up by itself, in the order of its chunks).  A CTA takes a run
// and 32 W columns; its kJoinParts warps each add a stretch of the run's pieces,
// and the first warp the stretches.
constexpr int kJoinParts = 8;
template <int W>
__global__ void __launch_bounds__(32 * kJoinParts) embed_join_kernel(const SumArgs p) {
  __shared__ float sums[kJoinParts][32 * W];
  wait_for_launch_before();
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int slabs = (p.H + 32 * W - 1) / (32 * W);
  const long long items = static_cast<long long>(*p.n_runs) * slabs;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int run = static_cast<int>(item / slabs);
    const int c = (static_cast<int>(item - static_cast<long long>(run) * slabs) * 32 + lane) * W;
    const int first = p.runs[run];
    const int key = p.keys[(static_cast<long long>(first) + 1) * p.chunk - 1];
    // the run's last chunk: the last that begins with its id
    int last = first + 1, end = p.n_chunks;
    while (end - last > 1) {
      const int step = (end - last + 31) / 32;
      const long long probe = last + (lane + 1ll) * step;
      const bool in = probe < end && p.keys[probe * p.chunk] == key;
      last += __popc(__ballot_sync(0xffffffffu, in)) * step;
      end = end < last + step ? end : last + step;
    }
    const int pieces = last - first + 1;
    const int per = (pieces + kJoinParts - 1) / kJoinParts;
    const int to = (part + 1) * per < pieces ? (part + 1) * per : pieces;
    float acc[W] = {};
    if (c < p.H) {
#pragma unroll 8
      for (int q = part * per; q < to; ++q) {
        const float* from = p.partial + (q == 0 ? 2ll * first + 1 : 2ll * (first + q)) * p.H + c;
        float f[W];
        widen<float, W>(load_raw<float, W>(from), f);   // written by the launch before
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] += f[i];
      }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) sums[part][lane * W + i] = acc[i];
    __syncthreads();
    if (part == 0 && c < p.H) {
      for (int q = 1; q < kJoinParts; ++q)
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] += sums[q][lane * W + i];
      put_row<W>(p.dw + static_cast<long long>(key) * p.H + c, acc, p.scale, p.accumulate);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- short lists

// Up to kFewTokens tokens: one launch, no sorted list.  A CTA is a token and a
// stretch of columns; it ends at once if an earlier token has its id, and else
// lists the tokens that have it, in their order, and sums them (blockDim.y
// stretches of the list where the columns leave threads for that).  The CTAs
// after them fill the other rows.  CTA 0 also checks the ids and writes the
// status word.  An id that all tokens name is one CTA's work; that is why the
// lists end at 512.
constexpr int kFewTokens = 512;

template <typename T, int VEC>
__global__ void __launch_bounds__(kSumThreads)
embed_few_kernel(const SumArgs p, const int* __restrict__ ids, DevStatus* st) {
  constexpr int U = 2 * kSumUnroll<VEC>, M = kCols<VEC>;
  __shared__ int list[kFewTokens];
  __shared__ int warp_n[kSumThreads / 32];
  __shared__ int first_bad;
  __shared__ float sums[kSumThreads * VEC * M];
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = static_cast<int>(p.T);
  if (blockIdx.x == 0) {
    if (tid == 0) first_bad = n;
    __syncthreads();
    for (int j = tid; j < n; j += kSumThreads)
      if (ids[j] < -1 || ids[j] >= p.V) atomicMin(&first_bad, j);
    __syncthreads();
    if (tid == 0) {
      const bool bad = first_bad < n;
      st->code = bad ? kStInvalidArg : kStOk;
      st->where = bad ? kWhereEmbed : 0;
      st->info = bad ? first_bad : 0;
    }
  }
  if (blockIdx.x >= p.sum_ctas) {
    if (p.accumulate) return;           // an empty list: only the status
    const long long v0 = static_cast<long long>(blockIdx.x - p.sum_ctas) * p.zero_rows;
    if (tid < p.zero_rows) list[tid] = v0 + tid >= p.V;
    __syncthreads();
    for (int j = tid; j < n; j += kSumThreads) {
      const long long r = ids[j] - v0;
      if (r >= 0 && r < p.zero_rows) list[r] = 1;
    }
    __syncthreads();
    zero_rows(p, v0, list, tid);
    return;
  }
  const int step = blockDim.x * VEC, width = M * step;
  const int slabs = (p.H + width - 1) / width;
  const int t = blockIdx.x / slabs, slab = blockIdx.x - t * slabs;
  const int id = ids[t];
  if (id < 0 || id >= p.V) return;
  int count = 0;
  for (int j0 = 0; j0 < n; j0 += kSumThreads) {
    const int j = j0 + tid;
    const bool same = j < n && ids[j] == id;
    const unsigned m = __ballot_sync(0xffffffffu, same);
    if (lane == 0) warp_n[warp] = __popc(m);
    if (__syncthreads_or(same && j < t)) return;
    int at = count + __popc(m & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kSumThreads / 32; ++w) {
      if (w < warp) at += warp_n[w];
      count += warp_n[w];
    }
    if (same) list[at] = j;
    __syncthreads();
  }
  const int c = slab * width + threadIdx.x * VEC;
  const int per = (count + blockDim.y - 1) / blockDim.y;
  const int to = static_cast<int>(threadIdx.y + 1) * per < count ? (threadIdx.y + 1) * per : count;
  float acc[M][VEC] = {};
  if (c < p.H) {
    const T* dout = static_cast<const T*>(p.dout) + c;
    for (int i = threadIdx.y * per; i < to; i += U) {
      Raw<T, VEC> raw[U][M];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < M; ++m)
          if (i + u < to && c + m * step < p.H)
            raw[u][m] = load_const<T, VEC>(dout + static_cast<long long>(list[i + u]) * p.H + m * step);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < M; ++m)
          if (i + u < to && c + m * step < p.H) {
            float f[VEC];
            widen<T, VEC>(raw[u][m], f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[m][e] += f[e];
          }
    }
  }
  if (blockDim.y > 1) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int e = 0; e < VEC; ++e) sums[(m * VEC + e) * kSumThreads + tid] = acc[m][e];
    __syncthreads();
    if (threadIdx.y > 0) return;
    for (int y = 1; y < static_cast<int>(blockDim.y); ++y)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[m][e] += sums[(m * VEC + e) * kSumThreads + y * blockDim.x + tid];
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
    if (c + m * step < p.H)
      put_row<VEC>(p.dw + static_cast<long long>(id) * p.H + c + m * step, acc[m], p.scale, p.accumulate);
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
  s.sum_ctas = 0;
  s.n_runs = run_count(a.status);
  s.runs = reinterpret_cast<int*>(a.scratch + pl.runs);
  s.n_chunks = static_cast<int>((a.T + pl.chunk - 1) / pl.chunk);
  // 128 KB of dw a CTA, less where that would leave the machine idle
  long long rows = 32768 / a.H;
  if (rows > a.V / 1024) rows = a.V / 1024;
  s.zero_rows = static_cast<int>(rows < 4 ? 4 : rows > kSumThreads ? kSumThreads : rows);
  return s;
}

int sort_passes(int V) {
  int bits = 1;
  while (bits < 31 && (V >> bits) != 0) ++bits;   // keys 0 .. V
  return (bits + kSortBits - 1) / kSortBits;
}

}  // namespace

template <typename T, int VEC>
static cudaError_t embed_fwd_t(const EmbedFwdArgs& a, int num_sms, cudaStream_t s) {
  if (a.status) {
    const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(DevStatus), s);
    if (e != cudaSuccess || a.T == 0) return e;
  }
  int tx = 32;
  while (tx < 256 && tx * VEC < a.H) tx *= 2;
  const dim3 block(tx, 256 / tx);
  // four rows a thread once that still fills the machine ([65536, 5120] bf16,
  // Zipf-distributed ids: 130 us against 139 with one)
  const long long groups = (a.T + 4 * block.y - 1) / (4 * block.y);
  if (groups >= 8LL * num_sms) {
    embed_fwd_kernel<T, VEC, 4><<<static_cast<unsigned>(groups), block, 0, s>>>(a);
  } else {
    const long long grid = (a.T + block.y - 1) / block.y;
    embed_fwd_kernel<T, VEC, 1><<<static_cast<unsigned>(grid), block, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, int is_bf16, int num_sms, cudaStream_t s) {
  if (is_bf16)
    return a.H % 8 == 0 ? embed_fwd_t<__nv_bfloat16, 8>(a, num_sms, s)
                        : embed_fwd_t<__nv_bfloat16, 1>(a, num_sms, s);
  return a.H % 4 == 0 ? embed_fwd_t<float, 4>(a, num_sms, s) : embed_fwd_t<float, 1>(a, num_sms, s);
}

// A chunk is as long as leaves 4096 pairs of a chunk and 512 columns, 16 to 128
// tokens: short chunks keep small calls parallel, long ones keep the pieces of runs
// few.  (A CTA of the sums takes 512 columns in fp32 and in rows of odd width, 1024
// in bf16: half as many CTAs there.)
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
  p.runs = o; o = up(o + 4 * chunks);
  p.total = o;
  return p;
}

// Threads of a row and rows (or stretches) of a CTA of kSumThreads.
template <int VEC>
static dim3 sum_block(int H, int least) {
  int tx = least;
  while (tx < kSumThreads && tx * VEC * kCols<VEC> < H) tx *= 2;
  return dim3(tx, kSumThreads / tx);
}

template <int VEC>
static long long sum_slabs(int H, const dim3& block) {
  const long long width = static_cast<long long>(block.x) * VEC * kCols<VEC>;
  return (H + width - 1) / width;
}

static long long zero_ctas(const SumArgs& s) {
  return s.accumulate ? 0 : (static_cast<long long>(s.V) + s.zero_rows - 1) / s.zero_rows;
}

template <typename T, int VEC>
static cudaError_t few_t(SumArgs s, const EmbedBwdArgs& a, cudaStream_t st) {
  const dim3 block = sum_block<VEC>(s.H, 16);
  s.sum_ctas = static_cast<int>(s.T * sum_slabs<VEC>(s.H, block));
  const long long grid = s.sum_ctas + zero_ctas(s);
  embed_few_kernel<T, VEC><<<static_cast<unsigned>(grid > 0 ? grid : 1), block, 0, st>>>(s, a.ids, a.status);
  return cudaGetLastError();
}

bool embed_bwd_sorts(long long T) { return T > kFewTokens; }

template <int kRounds>
static cudaError_t cluster_sort(const ClusterSort& p, cudaStream_t s) {
  const int smem = kClusterThreads * kRounds * static_cast<int>(sizeof(int2)) +
                   kClusterWarps * kSortBins * static_cast<int>(sizeof(short));
  const cudaError_t e = allow_smem<cluster_sort_kernel<kRounds>>(smem);
  if (e != cudaSuccess) return e;
  cluster_sort_kernel<kRounds><<<kClusterCtas, kClusterThreads, smem, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_embed_sort(const EmbedBwdArgs& a, cudaStream_t s) {
  const EmbedBwdPlan pl = embed_bwd_plan(a.T, a.H, a.V);
  const int passes = sort_passes(a.V);
  if (a.T <= kClusterMost) {
    ClusterSort p;
    p.ids = a.ids;
    p.keys_out = reinterpret_cast<int*>(a.scratch + pl.keys[(passes - 1) & 1]);
    p.pos_out = reinterpret_cast<int*>(a.scratch + pl.pos[(passes - 1) & 1]);
    p.T = a.T;
    p.V = a.V;
    p.passes = passes;
    p.status = a.status;
    const long long per = 1ll * kClusterCtas * kClusterThreads;
    return a.T <= per ? cluster_sort<1>(p, s)
                      : a.T <= 2 * per ? cluster_sort<2>(p, s) : cluster_sort<4>(p, s);
  }
  cudaError_t e = cudaMemsetAsync(a.status, 0, kClearBytes, s);
  if (e != cudaSuccess) return e;
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
    if (i == 0) {
      sort_hist_kernel<<<p.n_tiles, kSortThreads, 0, s>>>(p);
      e = cudaGetLastError();
    } else {
      e = launch_overlapped(sort_hist_kernel, dim3(p.n_tiles), dim3(kSortThreads), 0, s, p);
    }
    if (e == cudaSuccess)
      e = launch_overlapped(sort_scatter_kernel, dim3(p.n_tiles), dim3(kSortThreads), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int VEC>
static cudaError_t sum_t(SumArgs s, cudaStream_t st) {
  const dim3 block = sum_block<VEC>(s.H, 32);
  s.sum_ctas = static_cast<int>((s.n_chunks + block.y - 1) / block.y * sum_slabs<VEC>(s.H, block));
  return launch_overlapped(embed_sum_kernel<T, VEC>,
                           dim3(static_cast<unsigned>(s.sum_ctas + zero_ctas(s))), block, 0, st, s);
}

cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, int is_bf16, int num_sms, cudaStream_t st) {
  const EmbedBwdPlan pl = embed_bwd_plan(a.T, a.H, a.V);
  const SumArgs s = sum_args(a, pl, (sort_passes(a.V) - 1) & 1);
  const bool aligned = a.H % (is_bf16 ? 8 : 4) == 0;
  if (!embed_bwd_sorts(a.T)) {
    if (is_bf16) return aligned ? few_t<__nv_bfloat16, 8>(s, a, st) : few_t<__nv_bfloat16, 1>(s, a, st);
    return aligned ? few_t<float, 4>(s, a, st) : few_t<float, 1>(s, a, st);
  }
  cudaError_t e;
  if (is_bf16) e = aligned ? sum_t<__nv_bfloat16, 8>(s, st) : sum_t<__nv_bfloat16, 1>(s, st);
  else e = aligned ? sum_t<float, 4>(s, st) : sum_t<float, 1>(s, st);
  if (e != cudaSuccess || s.n_chunks <= 2) return e;   // no run of three chunks
  const int w = a.H % 4 == 0 ? 4 : 1;
  const long long most = static_cast<long long>(s.n_chunks) * ((a.H + 32 * w - 1) / (32 * w));
  // an item is a chain of latencies, so as many at a time as there may be
  const dim3 grid(static_cast<unsigned>(most < 64LL * num_sms ? most : 64LL * num_sms));
  return w == 4 ? launch_overlapped(embed_join_kernel<4>, grid, dim3(32 * kJoinParts), 0, st, s)
                : launch_overlapped(embed_join_kernel<1>, grid, dim3(32 * kJoinParts), 0, st, s);
}

}  // namespace eas
