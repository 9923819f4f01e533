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

// CTA 0 also checks every id and writes the status word: no other launch clears
// it.
template <typename T, int VEC, int kRows>
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
  // kRows rows a thread: their ids come in one latency and their loads leave
  // together
  const long long t0 = (static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y) * kRows;
  const T* src[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int id = t0 + r < p.T ? p.ids[t0 + r] : -1;
    src[r] = id >= 0 && id < p.V ? static_cast<const T*>(p.table) + static_cast<long long>(id) * p.H : nullptr;
  }
  T* dst = static_cast<T*>(p.out) + t0 * p.H;
#pragma unroll 4
  for (int c = threadIdx.x * VEC; c < p.H; c += blockDim.x * VEC) {
    Raw<T, VEC> raw[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (src[r]) raw[r] = load_raw<T, VEC>(src[r] + c);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (t0 + r >= p.T) break;
      float f[VEC] = {};
      if (src[r]) {
        widen<T, VEC>(raw[r], f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] *= p.scale;
      }
      // the table's rows come again, the output does not: 128 us against 136 at
      // [65536, 5120] bf16 with Zipf-distributed ids
      store_vec<T, VEC, true>(dst + static_cast<long long>(r) * p.H + c, f);
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
// meanwhile, so one buffer is enough.
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

// Zeros in the n floats at p by the CTA's kSumThreads threads; p need not start on
// a 16-byte boundary (rows of odd width).
__device__ __forceinline__ void zero_floats(float* p, int n, int tid) {
  int head = static_cast<int>(-(reinterpret_cast<uintptr_t>(p) >> 2) & 3);
  if (head > n) head = n;
  const int mid = (n - head) & ~3;
  for (int c = tid * 4; c < mid; c += kSumThreads * 4)
    *reinterpret_cast<float4*>(p + head + c) = make_float4(0.f, 0.f, 0.f, 0.f);
  if (tid < n - mid) p[tid < head ? tid : mid + tid] = 0.f;
}

// Zeros in rows [v0, v0 + p.zero_rows) of dw, but for those that a token names:
// each row's id is looked up in the sorted list.
__device__ __forceinline__ void zero_rows(const SumArgs& p, int block, int* skip) {
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
  for (int r = 0; r < p.zero_rows; ++r)
    if (!skip[r]) zero_floats(p.dw + (v0 + r) * p.H, p.H, tid);
}

// CTA b < p.sum_ctas: blockDim.y chunks of the sorted tokens (one where the
// columns fill the CTA), blockDim.x * VEC columns of them.  The CTAs after them fill the rows that no token names, so that
// their stores run beside the others' loads.
template <typename T, int VEC>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const SumArgs p) {
  __shared__ int key_store[4][kMaxChunk + 2];
  __shared__ int pos_store[4][kMaxChunk];
  wait_for_launch_before();
  if (blockIdx.x >= p.sum_ctas) {
    zero_rows(p, blockIdx.x - p.sum_ctas, key_store[0]);
    return;
  }
  int* keys = key_store[threadIdx.y];   // [0]: the key before the chunk, [n + 1]: the one after
  int* pos = pos_store[threadIdx.y];
  const int slabs = (p.H + blockDim.x * VEC - 1) / (blockDim.x * VEC);
  const int group = blockIdx.x / slabs, slab = blockIdx.x - group * slabs;
  const int chunk = group * blockDim.y + threadIdx.y;
  const long long i0 = static_cast<long long>(chunk) * p.chunk;
  const long long left = p.T - i0;
  const int n = static_cast<int>(left < 0 ? 0 : left < p.chunk ? left : p.chunk);
  for (int i = threadIdx.x; i < n + 2; i += blockDim.x) {
    const long long k = i0 + i - 1;
    keys[i] = k >= 0 && k < p.T ? p.keys[k] : -1;
    if (i < n) pos[i] = p.pos[i0 + i];
  }
  __syncthreads();
  const int c = (slab * blockDim.x + threadIdx.x) * VEC;
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
            float* q = p.partial + (2ll * chunk + (from_before ? 0 : 1)) * p.H + c;
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
  wait_for_launch_before();
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

// ------------------------------------------------------------- short lists

// Up to kFewTokens tokens: one launch, no sorted list.  A CTA is a token and
// kSumThreads * VEC columns; it ends at once if an earlier token has its id, and
// else lists the tokens that have it, in their order, and sums them.  The CTAs
// after them fill the other rows.  CTA 0 also checks the ids and writes the
// status word.  An id that all of 512 tokens name is one CTA's work (about 50
// us); that is why the lists end there.
constexpr int kFewTokens = 512;

template <typename T, int VEC>
__global__ void __launch_bounds__(kSumThreads)
embed_few_kernel(const SumArgs p, const int* __restrict__ ids, DevStatus* st) {
  __shared__ int list[kFewTokens];
  __shared__ int warp_n[kSumThreads / 32];
  __shared__ int first_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    for (int r = 0; r < p.zero_rows; ++r)
      if (!list[r]) zero_floats(p.dw + (v0 + r) * p.H, p.H, tid);
    return;
  }
  const int slabs = (p.H + kSumThreads * VEC - 1) / (kSumThreads * VEC);
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
  const int c = (slab * kSumThreads + tid) * VEC;
  if (c >= p.H) return;
  const T* dout = static_cast<const T*>(p.dout) + c;
  float acc[VEC] = {};
  for (int i = 0; i < count; i += kSumUnroll) {
    Raw<T, VEC> raw[kSumUnroll];
#pragma unroll
    for (int u = 0; u < kSumUnroll; ++u)
      if (i + u < count) raw[u] = load_raw<T, VEC>(dout + static_cast<long long>(list[i + u]) * p.H);
#pragma unroll
    for (int u = 0; u < kSumUnroll; ++u) {
      if (i + u < count) {
        float f[VEC];
        widen<T, VEC>(raw[u], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += f[e];
      }
    }
  }
  put_row<VEC>(p.dw + static_cast<long long>(id) * p.H + c, acc, p.scale, p.accumulate);
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
  const long long rows = 32768 / (a.H > 0 ? a.H : 1);   // 128 KB of dw
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
  int tx = 32;
  while (tx < 256 && tx * VEC < a.H) tx *= 2;
  const dim3 block(tx, 256 / tx);
  // four rows a thread once that still fills the machine ([65536, 5120] bf16:
  // 133 us against 139 with one)
  const long long groups = (a.T + 4 * block.y - 1) / (4 * block.y);
  if (groups >= 8LL * num_sms) {
    embed_fwd_kernel<T, VEC, 4><<<static_cast<unsigned>(groups), block, 0, s>>>(a);
  } else {
    const long long grid = a.T > 0 ? (a.T + block.y - 1) / block.y : 1;
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

template <typename T, int VEC>
static cudaError_t few_t(SumArgs s, const EmbedBwdArgs& a, cudaStream_t st) {
  const long long slabs = (s.H + kSumThreads * VEC - 1) / (kSumThreads * VEC);
  const long long zeros = s.accumulate ? 0 : (static_cast<long long>(s.V) + s.zero_rows - 1) / s.zero_rows;
  s.sum_ctas = static_cast<int>(s.T * slabs);
  const long long grid = s.sum_ctas + zeros;
  embed_few_kernel<T, VEC><<<static_cast<unsigned>(grid > 0 ? grid : 1), kSumThreads, 0, st>>>(s, a.ids, a.status);
  return cudaGetLastError();
}

bool embed_bwd_sorts(long long T) { return T > kFewTokens; }

template <int kRounds>
static cudaError_t cluster_sort(const ClusterSort& p, cudaStream_t s) {
  const int smem = kClusterThreads * kRounds * static_cast<int>(sizeof(int2)) +
                   kClusterWarps * kSortBins * static_cast<int>(sizeof(short));
  const cudaError_t e = cudaFuncSetAttribute(cluster_sort_kernel<kRounds>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
  cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(DevStatus), s);
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
static cudaError_t sum_t(SumArgs s, int n_chunks, cudaStream_t st) {
  int tx = 32;
  while (tx < kSumThreads && tx * VEC < s.H) tx *= 2;
  const dim3 block(tx, kSumThreads / tx);
  const long long slabs = (s.H + tx * VEC - 1) / (tx * VEC);
  const long long zeros = s.accumulate ? 0 : (static_cast<long long>(s.V) + s.zero_rows - 1) / s.zero_rows;
  s.sum_ctas = static_cast<int>((n_chunks + block.y - 1) / block.y * slabs);
  return launch_overlapped(embed_sum_kernel<T, VEC>, dim3(static_cast<unsigned>(s.sum_ctas + zeros)),
                           block, 0, st, s);
}

cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, int is_bf16, cudaStream_t st) {
  const EmbedBwdPlan pl = embed_bwd_plan(a.T, a.H, a.V);
  const SumArgs s = sum_args(a, pl, (sort_passes(a.V) - 1) & 1);
  if (!embed_bwd_sorts(a.T)) {
    if (a.H % (is_bf16 ? 8 : 4) == 0)
      return is_bf16 ? few_t<__nv_bfloat16, 8>(s, a, st) : few_t<float, 4>(s, a, st);
    return is_bf16 ? few_t<__nv_bfloat16, 1>(s, a, st) : few_t<float, 1>(s, a, st);
  }
  const int n_chunks = static_cast<int>((a.T + pl.chunk - 1) / pl.chunk);
  const int vec16 = is_bf16 ? 8 : 4;
  cudaError_t e;
  if (a.H % vec16 == 0)
    e = is_bf16 ? sum_t<__nv_bfloat16, 8>(s, n_chunks, st) : sum_t<float, 4>(s, n_chunks, st);
  else
    e = is_bf16 ? sum_t<__nv_bfloat16, 1>(s, n_chunks, st) : sum_t<float, 1>(s, n_chunks, st);
  if (e != cudaSuccess || n_chunks <= 1) return e;
  return launch_overlapped(embed_join_kernel,
                           dim3(n_chunks, (a.H + kSumThreads - 1) / kSumThreads), dim3(kSumThreads),
                           0, st, s, n_chunks);
}

}  // namespace eas
