// Orthogonalised update of a matrix: momentum, then Newton-Schulz products.
//
//   m' = beta m + (1 - beta) g,  u = m' or (1 - beta) g + beta m',
//   X = u / (|u| + eps), transposed where it is taller than wide: [n][m], n <= m;
//   each step  A = X X^T,  B = b A + c A A,  X = a X + B X;  out = scale X.
//
// The products run on the tensor cores with fp16 operands and fp32 accumulators.
// X is kept in 22 bits: hi in fp16, and what that leaves out, lo, in fp16 too (times 2^11).
// hi is multiplied; B holds a on its diagonal, so B hi + a lo is the next X.  What decides
// the precision is X's own rounding: an error in directions that the gradient does not have
// grows by a each step, beside singular values near 1 that do not grow: 485 times in five of
// the usual steps, 20 000 times in eight.  A gradient of rank 1 in five steps ends 1.5e-1 off
// with hi alone, 7e-3 with lo in eight bits (e5m2), 2.6e-3 with these; rank 8 in seven steps
// 5e-1, 2.3e-2 and 2.5e-3 (256 x 512; the output's rounding to bf16 is 1.7e-3 of it).  lo in
// eight bits would save 2 to 4 % of the time at 1024 rows and more.  The roundings of A, B
// and of hi in the products stay where they are, each 2^-11 of its own product: they turn
// singular vectors, which does not grow.  fp32 sums leave 2^-23 of X a step for every 16 terms,
// in squares, and that does: about 3e-8 sqrt(n) prod |a|.  Everything is stored times 2^12, so
// that fp16's range covers entries from 2^-36 to 16.
//
// A and A A are symmetric: only tiles on and above the diagonal are computed, and
// stored twice, the second time transposed.  A step takes 3 n^2 m + n^3 operations.
#include <cstring>
#include <type_traits>

#include <cuda_fp16.h>

#include "eas_launch.cuh"
#include "eas_mma.cuh"
#include "eas_ops.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr float kUp = 4096.f, kDown = 1.f / 4096.f;   // the stored scale
constexpr float kLoUp = 2048.f, kLoDown = 1.f / 2048.f;
constexpr int kWhereMuon = 50;

// ------------------------------------------------- momentum, norm, conversion

constexpr int kPrepThreads = 256;
constexpr int kChunk = 4096;      // elements a CTA at least
constexpr int kMostChunks = 1024; // partial sums a matrix

// Whether a sum of squares is as good in fp32 as its roundings: it has not come near the
// ends of fp32's range.
__device__ __forceinline__ bool in_range(float s) { return s > 1e-30f && s < 1e30f; }

// Sum of squares in fp64, added up in fp32 over the values of a call where that is safe
// (an fp64 operation costs 32 of fp32).
template <int K, int VEC>
__device__ __forceinline__ double squares(const float (&u)[K][VEC]) {
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s = fmaf(u[k][j], u[k][j], s);
  if (in_range(s)) return s;
  double d = 0.;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < VEC; ++j) d += static_cast<double>(u[k][j]) * u[k][j];
  return d;
}

// VEC consecutive values: one, or 16-byte vectors of them.
template <typename T, int VEC>
__device__ __forceinline__ void read_values(const T* p, float (&f)[VEC]) {
  constexpr int W = VEC == 1 ? 1 : kVec16<T>;
#pragma unroll
  for (int h = 0; h < VEC; h += W) {
    float part[W];
    widen<T, W>(load_raw<T, W>(p + h), part);
#pragma unroll
    for (int j = 0; j < W; ++j) f[h + j] = part[j];
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void write_values(T* p, const float (&f)[VEC]) {
  constexpr int W = VEC == 1 ? 1 : kVec16<T>;
#pragma unroll
  for (int h = 0; h < VEC; h += W) {
    float part[W];
#pragma unroll
    for (int j = 0; j < W; ++j) part[j] = f[h + j];
    store_vec<T, W>(p + h, part);
  }
}

// The update u of VEC values (and the new momentum in m): in one place, so that the norm
// and X see the same bits.
template <int VEC>
__device__ __forceinline__ void update_of(const MuonArgs& a, const float (&g)[VEC], float (&m)[VEC], float (&u)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    m[j] = fmaf(a.beta, m[j], a.rest * g[j]);
    u[j] = a.nesterov ? fmaf(a.beta, m[j], a.rest * g[j]) : m[j];
  }
}

// The updates of groups of values, in place of the gradients.
template <int K, int VEC>
__device__ __forceinline__ void updates_of(const MuonArgs& a, float (&g)[K][VEC], float (&m)[K][VEC]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float u[VEC];
    update_of<VEC>(a, g[k], m[k], u);
#pragma unroll
    for (int j = 0; j < VEC; ++j) g[k][j] = u[j];
  }
}

// Sum of squares of a chunk of a matrix's update.  A thread has kItems vectors (kVec) or
// single values on their way at a time.
template <typename G, typename M, bool kMom, bool kVec>
__device__ double chunk_squares(const MuonArgs& a, long long base, long long lo, long long hi) {
  constexpr int VEC = kVec ? 8 : 1, kItems = kVec ? 2 : 8;
  const G* grad = static_cast<const G*>(a.grad) + base;
  const M* mom = static_cast<const M*>(a.mom) + base;
  double sum = 0.;
  for (long long i0 = lo + static_cast<long long>(threadIdx.x) * VEC; i0 < hi; i0 += kItems * kPrepThreads * VEC) {
    float g[kItems][VEC] = {};
    [[maybe_unused]] float m[kItems][VEC] = {};
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const long long i = i0 + k * kPrepThreads * VEC;
      if (i >= hi) break;
      read_values(grad + i, g[k]);
      if constexpr (kMom) read_values(mom + i, m[k]);
    }
    if constexpr (kMom) updates_of(a, g, m);
    sum += squares(g);
  }
  return sum;
}

// Sum over the CTA of kN threads, in thread 0.
template <int kN>
__device__ double block_sum(double v) {
  __shared__ double part[kN / 32];
  float f = static_cast<float>(v);
  if (__all_sync(0xffffffffu, v == 0. || in_range(f))) {      // squares: their sum stays below 32 * 1e30
#pragma unroll
    for (int d = 16; d; d >>= 1) f += __shfl_down_sync(0xffffffffu, f, d);
    v = f;
  } else {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_down_sync(0xffffffffu, v, d);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.;
    for (int w = 0; w < kN / 32; ++w) v += part[w];
  }
  return v;
}

// grid (chunks, L)
template <typename G, typename M, bool kMom>
__global__ void __launch_bounds__(kPrepThreads) muon_norm_kernel(const MuonArgs a) {
  const long long size = static_cast<long long>(a.rows) * a.cols, base = blockIdx.y * size;
  const long long lo = blockIdx.x * a.chunk, hi = lo + a.chunk < size ? lo + a.chunk : size;
  bool vec = (size & 7) == 0 && aligned16(a.grad);
  if constexpr (kMom) vec = vec && aligned16(a.mom);
  const double sum = block_sum<kPrepThreads>(vec ? chunk_squares<G, M, kMom, true>(a, base, lo, hi)
                                   : chunk_squares<G, M, kMom, false>(a, base, lo, hi));
  if (threadIdx.x == 0) {
    a.partial[blockIdx.y * gridDim.x + blockIdx.x] = sum;
    if (blockIdx.x == 0 && blockIdx.y == 0) *a.status = DevStatus{0, 0, 0, 0};
  }
  // the products' counters
  const long long cta = static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x;
  for (long long i = cta * kPrepThreads + threadIdx.x; i < a.sync_words;
       i += static_cast<long long>(gridDim.x) * gridDim.y * kPrepThreads)
    a.sync[i] = 0;
}

// A value's hi and lo: pairs of them.
__device__ __forceinline__ uint32_t hi_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 hi_values(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t lo_bits(float a, float b, uint32_t hi) {
  const float2 h = hi_values(hi);
  return hi_bits((a - h.x) * kLoUp, (b - h.y) * kLoUp);
}

__device__ __forceinline__ void write_pair(const MuonPair& x, long long o, const float (&v)[8], float f) {
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float p = v[2 * j] * f, q = v[2 * j + 1] * f;
    hi[j] = hi_bits(p, q);
    lo[j] = lo_bits(p, q, hi[j]);
  }
  *reinterpret_cast<uint4*>(x.hi + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(x.lo + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// 2^12 / (norm + eps) from the sum of squares.
__device__ __forceinline__ float factor_of(double sum, float eps) {
  const float s = static_cast<float>(sum);
  if (in_range(s)) return kUp / (sqrtf(s) + eps);
  return static_cast<float>(kUp / (sqrt(sum) + eps));
}

// The new momentum, and X's first pair: the update times 2^12 / (norm + eps), transposed
// where it is taller than wide.  grid (CTAs, L); a CTA takes 64 x 64 tiles of X in turn.
template <typename G, typename M, bool kMom, bool kTall>
__global__ void __launch_bounds__(kPrepThreads) muon_scale_kernel(const MuonArgs a) {
  __shared__ float tile[kTall ? 64 : 1][65];
  __shared__ float factor;
  const int tid = threadIdx.x;
  const long long l = blockIdx.y, base = l * a.rows * a.cols;
  const G* grad = static_cast<const G*>(a.grad) + base;
  const M* mom = static_cast<const M*>(a.mom) + base;
  M* new_mom = static_cast<M*>(a.new_mom) + base;
  wait_for_launch_before();
  double s = 0.;
  for (int i = tid; i < a.chunks; i += kPrepThreads) s += a.partial[l * a.chunks + i];
  s = block_sum<kPrepThreads>(s);
  if (tid == 0) factor = factor_of(s, a.eps);
  __syncthreads();
  const float f = factor;
  const int across = (a.m + 63) / 64, tiles = across * ((a.n + 63) / 64);
  // rows of the source in vectors of eight
  const bool vec = (a.cols & 7) == 0 && aligned16(grad) && (!kMom || (aligned16(mom) && aligned16(new_mom)));
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int r0 = t / across * 64, c0 = t % across * 64;      // of X
    // a tile is 64 rows of eight vectors of the source: two a thread
    float v[2][8], m[2][8];
    long long at[2];
    int left[2];                                               // of the row, from there on
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = k * kPrepThreads + tid;
      const int sr = (kTall ? c0 : r0) + i / 8, sc = (kTall ? r0 : c0) + i % 8 * 8;
      at[k] = static_cast<long long>(sr) * a.cols + sc;
      left[k] = sr < a.rows ? a.cols - sc : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = m[k][j] = 0.f;
      if (vec) {
        if (left[k] > 0) {
          read_values(grad + at[k], v[k]);
          if constexpr (kMom) read_values(mom + at[k], m[k]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left[k]) {
            v[k][j] = to_f32(grad[at[k] + j]);
            if constexpr (kMom) m[k][j] = to_f32(mom[at[k] + j]);
          }
      }
    }
    if constexpr (kMom) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float u[8];
        update_of<8>(a, v[k], m[k], u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = u[j];
        if (vec) {
          if (left[k] > 0) write_values(new_mom + at[k], m[k]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left[k]) {
              const float one[1] = {m[k][j]};
              store_vec<M, 1>(new_mom + at[k] + j, one);
            }
        }
      }
    }
    if constexpr (kTall) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = k * kPrepThreads + tid;
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[i / 8][i % 8 * 8 + j] = v[k][j];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = k * kPrepThreads + tid;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = tile[i % 8 * 8 + j][i / 8];
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = k * kPrepThreads + tid, r = r0 + i / 8;
      if (r < a.n) write_pair(a.x[0], (l * a.n + r) * a.ldx + c0 + i % 8 * 8, v[k], f);
    }
  }
}

// ------------------------------------------------------------------ products
//
// All products of all steps run in one launch.  Their tiles form one list (step by
// step: the tiles of A, of B, of X; each for all L matrices) that the CTAs draw from in
// order; a tile waits, 128 or 256 k at a time, for the tiles of earlier products that
// hold its operands.  Each tile has a counter for that: its storing warps add one when
// their stores are visible.  So the last tiles of a product and the first of the next
// one run side by side, and nothing is launched in between.  [4096][4096] takes 1.79 +
// 1.79 + 3.37 rounds of 76 tiles a step instead of 2 + 2 + 4.  Where A has few tiles and k
// is long, each is computed in parts; a warp that brings the last part of its slice adds
// the parts up, in their order.
//
// No CTA waits for a tile that no running CTA has drawn, since tiles are drawn in
// order and depend on earlier ones alone.  What a tile overwrites has no reader left
// when its operands are there: A(i, j) of a step needs rows i and j of X, those need
// rows i and j of the B before, and those all readers of the A(i, j) before; B and X
// likewise.

enum Kind { kGram, kPoly, kApply, kLast };

constexpr int kStoreWarps = 8;                     // at most
constexpr int kStages = 5;
constexpr int kRing = 3;                           // tile numbers on their way to the warps
constexpr int kOperand = 16384;                    // 128 rows (columns) x 64 k
constexpr int kEpiWarp = 8192;                     // two boxes a warp
constexpr int kSmem = kStages * 2 * kOperand + kStoreWarps * kEpiWarp + 1024 + 512;
constexpr int kDrawAhead = 6;                      // k-blocks before a tile's end
constexpr int kBand = 4;                           // rows of tiles of X that are computed together

// CG = 2: a pair of CTAs computes 256 x 256 tiles, each 128 of the rows; CG = 1: a CTA
// 128 x 128 tiles, or (kHalves = 2) each half of their columns on its own.
template <int CG, int kHalves>
struct Geo {
  static constexpr int kM = 128 * CG, kTile = 128 * CG;
  static constexpr int kN = kTile / kHalves;
  static constexpr int kRowsB = 128 / kHalves;     // of the second operand that a CTA loads
  static constexpr uint32_t kCols = 2 * kN;        // two accumulators
  static constexpr int kChunk = 2 * CG;            // k-blocks of 64 in a tile's width
  static constexpr int kStore = kStoreWarps / kHalves;
  static constexpr int kThreads = 96 + 32 * kStore;
  static constexpr int kDone = kStoreWarps * CG;   // arrivals that finish a tile, its halves together
};

struct GemmArgs {
  CUtensorMap xk[2], xs[2], xn[2], xh[2], xl[2];   // X's pairs: rows as first and second operand, columns as operand, stores
  CUtensorMap ak, a2, as, at, bk, bs, bt;   // A and B: first and second operand, store, transposed store
  int n, m, L, steps;
  int num_m, num_n;                         // tiles down and across X
  int tri, full;                            // tiles of A (or B), of X, a matrix
  int split, depth;                         // parts of a tile of A along k, and k-blocks of one
  float* parts;                             // [L][tri][8 slices of 32 x 64][split][64][32]
  int* arrived;                             // [L][tri][8]: parts of a slice that are there
  float coeffs[3 * kMuonSteps];
  __nv_bfloat16* out;
  float scale;
  int tall;
  int* counter;                             // next tile
  int* done_a;                              // [L][num_m][num_m], upper triangle
  int* done_b;
  int* done_x;                              // [L][num_m][num_n]
  DevStatus* status;
  long long budget;
};

struct Tile {
  int kind, step, l, m, n, half, part;
};

template <int kHalves>
__device__ __forceinline__ Tile tile_of(int t, const GemmArgs& a) {
  Tile w;
  w.half = t % kHalves;
  t /= kHalves;
  const int gram = a.L * a.tri * a.split, per_step = gram + a.L * (a.tri + a.full);
  w.step = t / per_step;
  t -= w.step * per_step;
  w.part = 0;
  if (t < gram + a.L * a.tri) {
    if (t < gram) {
      w.kind = kGram;
      w.part = t % a.split;
      t /= a.split;
    } else {
      w.kind = kPoly;
      t -= gram;
    }
    w.l = t / a.tri;
    t -= w.l * a.tri;
    // column by column of the upper triangle: n (n + 1) / 2 tiles before column n
    int n = static_cast<int>((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
    while (n * (n + 1) / 2 > t) --n;
    while ((n + 1) * (n + 2) / 2 <= t) ++n;
    w.n = n;
    w.m = t - n * (n + 1) / 2;
  } else {
    w.kind = w.step + 1 < a.steps ? kApply : kLast;
    t -= gram + a.L * a.tri;
    w.l = t / a.full;
    t -= w.l * a.full;
    // bands of rows, column by column: the next step's first tiles need the first
    // rows alone, and a band's tiles share X's columns
    const int band = t / (kBand * a.num_n), height = min(kBand, a.num_m - band * kBand);
    t -= band * kBand * a.num_n;
    w.n = t / height;
    w.m = band * kBand + t - w.n * height;
  }
  return w;
}

// A tile's k-blocks, from w.part * a.depth on.
__device__ __forceinline__ int k_blocks(const Tile& w, const GemmArgs& a) {
  const int all = ((w.kind == kGram ? a.m : a.n) + 63) / 64;
  return w.kind == kGram ? min(a.depth, all - w.part * a.depth) : all;
}

__device__ __forceinline__ int acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void release_add(int* p) {
  asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory");
}
// Orders this thread's acquired or released values with its TMA loads or stores.
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// How far a CTA's it-th tile has its operands: `chunks` of them.  Grows from tile to tile
// (and wraps around).
__device__ __forceinline__ uint32_t operands_to(int it, int chunks) { return (static_cast<uint32_t>(it) << 12) + chunks; }

// Counter of the operand that a tile reads at chunk c of k: its first operand's
// (which = 0) or its second one's.  null: none to wait for.
__device__ __forceinline__ const int* operand_counter(const Tile& w, int c, int which, const GemmArgs& a) {
  const int row = which ? w.n : w.m;
  if (which && (w.kind >= kApply || w.m == w.n)) return nullptr;   // Apply: B's row waits for all of X
  if (w.kind == kGram)
    return w.step ? a.done_x + static_cast<long long>(w.l) * a.full + row * a.num_n + c : nullptr;
  return (w.kind == kPoly ? a.done_a : a.done_b) + static_cast<long long>(w.l) * a.num_m * a.num_m +
         min(row, c) * a.num_m + max(row, c);
}

// 64 columns of this thread's accumulator row.
__device__ __forceinline__ void load64(uint32_t taddr, float (&v)[64]) {
  tmem_ld32(taddr, *reinterpret_cast<float(*)[32]>(&v[0]));
  tmem_ld32(taddr + 32, *reinterpret_cast<float(*)[32]>(&v[32]));
}

__device__ __forceinline__ uint32_t word_of(const uint4& r, int i) { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }

// 16-byte block j of a row in a [..][64] fp16 box in the 128-byte swizzled layout.
__device__ __forceinline__ uint4* swizzled(uint8_t* box, int row, int j) {
  return reinterpret_cast<uint4*>(box + row * 128 + ((j ^ (row & 7)) << 4));
}
__device__ __forceinline__ void get_box(uint8_t* box, int lane, uint4 (&r)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = *swizzled(box, lane, j);
}
__device__ __forceinline__ void put_box(uint8_t* box, int lane, const uint32_t (&w)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *swizzled(box, lane, j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// What a storing warp keeps: two boxes of 4 KB, their load barrier and its phase.  The first
// takes A and then A or B to be stored, the second their transpose.  Of X the second takes
// lo of the first 64 columns, then hi to be stored; the first lo of the other 64, then
// lo to be stored.
struct Boxes {
  uint8_t* box;
  uint64_t* bar;
  uint32_t phase;
};

// Lane 0: what the tile's columns from `col` on add to their products, to the warp's
// boxes: A's (64 columns) or lo (all `cols`).
template <int kKind>
__device__ __forceinline__ void fetch(const GemmArgs& a, const Tile& w, const Boxes& b, int row0, int col, int cols) {
  if constexpr (kKind == kPoly) {
    mbar_arrive_expect_tx(b.bar, 4096);
    mma::load_3d<1>(b.box, &a.as, smem_u32(b.bar), col, row0, w.l);
  } else if constexpr (kKind >= kApply) {
    const int n = min((a.m - col + 63) / 64, cols / 64);
    mbar_arrive_expect_tx(b.bar, 4096 * n);
    for (int c = 0; c < n; ++c)
      mma::load_3d<1>(b.box + 4096 * (1 - c), &a.xl[w.step & 1], smem_u32(b.bar), col + 64 * c, row0, w.l);
  }
}

// The parts of a slice of 32 rows and 64 columns of A: false for all but the last one to
// come, which gets their sum, in the order of the parts.
__device__ __forceinline__ bool sum_parts(const GemmArgs& a, const Tile& w, int slice, int lane, float (&v)[64]) {
  const long long s = (static_cast<long long>(w.l) * a.tri + w.n * (w.n + 1) / 2 + w.m) * kStoreWarps + slice;
  float* p = a.parts + s * a.split * 2048 + lane;
#pragma unroll
  for (int j = 0; j < 64; ++j) __stcg(p + w.part * 2048 + j * 32, v[j]);
  __threadfence();
  __syncwarp();
  int before = 0;
  if (lane == 0) before = atomicAdd(&a.arrived[s], 1);
  if (__shfl_sync(0xffffffffu, before, 0) != a.split - 1) return false;
  __threadfence();
  if (lane == 0) a.arrived[s] = 0;                 // for the next step, whose parts wait for this tile
#pragma unroll
  for (int j = 0; j < 64; ++j) v[j] = __ldcg(p + j * 32);
#pragma unroll 1
  for (int i = 1; i < a.split; ++i)
#pragma unroll
    for (int j = 0; j < 64; ++j) v[j] += __ldcg(p + i * 2048 + j * 32);
  return true;
}

// A warp's 32 rows (from row0 on; this thread's is row0 + lane) and kCols columns
// (from n0 on) of a tile.  What the first columns (lo: all) add has been fetched.  mine:
// whether the tile's counter is this warp's to add to (of a tile in parts, one does).
template <int kKind, int kCols>
__device__ __forceinline__ bool epilogue(const GemmArgs& a, const Tile& w, uint32_t tbase, int row0, int n0,
                                         int lane, Boxes& b, volatile int* abort_flag, int slice, bool& mine) {
  static_assert(kCols <= 128, "a box for lo of 64 columns each");
  const int width = kKind <= kPoly ? a.n : a.m;
  const int row = row0 + lane;
  const bool mirror = kKind <= kPoly && w.m != w.n;
  const int to = (w.step & 1) ^ 1;
  const float* abc = a.coeffs + 3 * w.step;
  uint8_t* box = b.box;
  uint4 lo[8];                                     // this row's of 64 columns
  constexpr int kUnroll = kKind >= kApply ? 2 : 1; // lo stays in registers
#pragma unroll kUnroll
  for (int c = 0; c < kCols / 64; ++c) {
    const int col = n0 + c * 64;
    if (col >= width || row0 >= a.n) break;        // the same for the warp
    if (c) {
      // the boxes have been read before they are filled again
      __syncwarp();
      if (lane == 0) {
        if constexpr (kKind != kLast) mma::stores_read();
        if constexpr (kKind == kPoly) fetch<kPoly>(a, w, b, row0, col, 64);
      }
    }
    float v[64];
    load64(tbase + c * 64, v);
    if (kKind == kPoly || (kKind >= kApply && c == 0)) {
      if (!mma::warp_wait(b.bar, b.phase, abort_flag, a.budget)) return false;
      b.phase ^= 1u;
    }
    if constexpr (kKind == kGram) {
      if (a.split > 1 && !(mine = sum_parts(a, w, slice, lane, v))) return true;
#pragma unroll
      for (int j = 0; j < 64; ++j) v[j] *= kDown;
    } else if constexpr (kKind == kPoly) {
      // a I + b A + c A A
      const float f = abc[1], g = abc[2] * kDown;
      uint4 r[8];
      get_box(box, lane, r);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 x = hi_values(word_of(r[j / 4], j % 4));
        v[2 * j] = fmaf(v[2 * j], g, f * x.x);
        v[2 * j + 1] = fmaf(v[2 * j + 1], g, f * x.y);
      }
      if (!mirror) {
        const int d = row - col;                   // the diagonal's place in the row
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] += j == d ? abc[0] * kUp : 0.f;
      }
    } else {
      // B hi + a lo
      const float f = abc[0] * kLoDown;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 r = kCols > 64 && c ? lo[j] : *swizzled(box + 4096, lane, j);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 x = hi_values(word_of(r, p));
          float* o = v + 8 * j + 2 * p;
          o[0] = fmaf(o[0], kDown, f * x.x);
          o[1] = fmaf(o[1], kDown, f * x.y);
        }
      }
    }
    // Last: the lanes write across the boxes' rows
    if constexpr (kKind == kLast && kCols > 64)
      if (c == 0) get_box(box, lane, lo);
    __syncwarp();                                  // lane 0 has waited for the box; lo and A have been read
    if constexpr (kKind == kLast) {
      const float up = a.scale * kDown;
      if (a.tall) {
        // X's rows are the output's columns: 32 lanes store 64 bytes in a row
        if (row < a.n) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (col + j < a.m)
              a.out[(static_cast<long long>(w.l) * a.m + col + j) * a.n + row] = __float2bfloat16_rn(v[j] * up);
        }
      } else {
        uint32_t* s = reinterpret_cast<uint32_t*>(box);      // [32][33] pairs
#pragma unroll
        for (int j = 0; j < 32; ++j) s[lane * 33 + j] = pack_bf16x2(v[2 * j] * up, v[2 * j + 1] * up);
        __syncwarp();
        const bool even = (a.m & 1) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 3u) == 0;
        const int cc = col + 2 * lane;
#pragma unroll 4
        for (int i = 0; i < 32; ++i) {
          if (row0 + i >= a.n) break;
          const uint32_t p = s[i * 33 + lane];
          __nv_bfloat16* o = a.out + (static_cast<long long>(w.l) * a.n + row0 + i) * a.m + cc;
          if (even) {
            if (cc < a.m) *reinterpret_cast<uint32_t*>(o) = p;
          } else {
            const __nv_bfloat162 q = *reinterpret_cast<const __nv_bfloat162*>(&p);
            if (cc < a.m) o[0] = q.x;
            if (cc + 1 < a.m) o[1] = q.y;
          }
        }
      }
    } else {
      if constexpr (kKind == kApply) {
        uint4 rest[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t h[4], l[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float x = v[8 * j + 2 * p], y = v[8 * j + 2 * p + 1];
            h[p] = hi_bits(x, y);
            l[p] = lo_bits(x, y, h[p]);
          }
          *swizzled(box + 4096, lane, j) = make_uint4(h[0], h[1], h[2], h[3]);
          rest[j] = make_uint4(l[0], l[1], l[2], l[3]);
        }
        // the other columns' lo waits in registers: its box is needed
        if (kCols > 64 && c == 0) get_box(box, lane, lo);
#pragma unroll
        for (int j = 0; j < 8; ++j) *swizzled(box, lane, j) = rest[j];
      } else {
        uint32_t hi[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) hi[j] = hi_bits(v[2 * j], v[2 * j + 1]);
        put_box(box, lane, hi);
        if (mirror) {
          // [64][32]: the columns as rows
          __half* t = reinterpret_cast<__half*>(box + 4096);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const __half2 h = *reinterpret_cast<const __half2*>(&hi[j]);
            t[(2 * j) * 32 + lane] = __low2half(h);
            t[(2 * j + 1) * 32 + lane] = __high2half(h);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kKind == kApply) {
          mma::store_3d(&a.xh[to], box + 4096, col, row0, w.l);
          mma::store_3d(&a.xl[to], box, col, row0, w.l);
        } else {
          mma::store_3d(kKind == kGram ? &a.as : &a.bs, box, col, row0, w.l);
          if (mirror) mma::store_3d(kKind == kGram ? &a.at : &a.bt, box + 4096, row0, col, w.l);
        }
        mma::store_commit();
      }
    }
  }
  return true;
}

// Warp 0 loads, warp 1 issues the MMAs, warps 2 to 9 store (two for each 32 rows, half of
// the columns each; 2 to 5 of a half tile), and the last warp draws the next tile and watches its operands'
// counters while this one's are loaded (the loads are what bounds a tile: 32 KB of
// operands for 512 clocks of MMA); two accumulators, so that a tile's stores run under the next
// one's products.
template <int CG, int kHalves>
__global__ void __launch_bounds__(Geo<CG, kHalves>::kThreads, 1) muon_gemm_kernel(const __grid_constant__ GemmArgs a) {
  using G = Geo<CG, kHalves>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* s_a = smem;
  uint8_t* s_b = smem + kStages * kOperand;
  uint8_t* s_epi = s_b + kStages * kOperand;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_epi + kStoreWarps * kEpiWarp);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* rfull = tempty + 2;
  uint64_t* rempty = rfull + kRing;
  uint64_t* there = rempty + kRing;        // of the tile in a ring slot: its operands
  uint64_t* fetched = there + kRing;       // of a storing warp: what it adds
  uint64_t* near_end = fetched + kStoreWarps;   // of the tile that is being loaded
  uint64_t* drain = near_end + 1;
  int* ring = reinterpret_cast<int*>(drain + 1);
  volatile uint32_t* progress = reinterpret_cast<volatile uint32_t*>(ring + kRing);   // see operands_to
  uint32_t* slot_addr = reinterpret_cast<uint32_t*>(ring + 2 * kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_addr + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = mma::rank_in_pair<CG>();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], G::kStore * CG);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&rfull[i], 1);
      mbar_init(&rempty[i], (2 + G::kStore) * CG);   // loader, MMA warp (CTA 1: drawer), storing warps
      mbar_init(&there[i], 1);
      progress[i] = 0;
    }
    for (int i = 0; i < G::kStore; ++i) mbar_init(&fetched[i], 1);
    mbar_init(near_end, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) mma::tmem_alloc<CG, G::kCols>(slot_addr);
  tc_fence_before();
  mma::sync_pair<CG>();
  tc_fence_after();
  const uint32_t tmem = *slot_addr;
  const int total = a.steps * a.L * (a.tri * a.split + a.tri + a.full) * kHalves;
  const uint32_t rempty0 = mma::leader_addr<CG>(&rempty[0]);

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t full0 = mma::leader_addr<CG>(&full[0]);
      for (int it = 0; ok; ++it) {
        const int slot = it % kRing;
        if (!mma::wait(&rfull[slot], (it / kRing) & 1, abort_flag, a.budget)) {
          report(a.status, kStTimeout, kWhereMuon, it);
          break;
        }
        const int t = ring[slot];
        mma::arrive_at(rempty0 + 8 * slot);
        if (t < 0) break;
        const Tile w = tile_of<kHalves>(t, a);
        const int from = w.step & 1;
        const CUtensorMap* ma = w.kind == kGram ? &a.xk[from] : w.kind == kPoly ? &a.ak : &a.bk;
        const CUtensorMap* mb = w.kind == kGram ? &a.xs[from] : w.kind == kPoly ? &a.a2 : &a.xn[from];
        const int mrow = w.m * G::kM + static_cast<int>(rank) * 128;
        const int ncol = w.n * G::kTile + w.half * G::kN + static_cast<int>(rank) * 128;
        const int num_kb = k_blocks(w, a);
        const int kb0 = w.part * a.depth;
        int known = 0;                       // k-blocks whose operands are there
        for (int kb = 0; kb < num_kb; ++kb) {
          if (kb == known) {
            const uint32_t want = operands_to(it, kb / G::kChunk + 1);
            const long long t0 = clock64();
            uint32_t have;
            while (static_cast<int>((have = progress[slot]) - want) < 0) {
              if (*abort_flag || clock64() - t0 > a.budget) {
                ok = false;
                break;
              }
            }
            if (!ok) {
              *abort_flag = 1;
              report(a.status, kStTimeout, kWhereMuon + 1, t);
              break;
            }
            __threadfence_block();
            fence_async_global();
            known = (kb / G::kChunk + 1 + static_cast<int>(have - want)) * G::kChunk;
          }
          if (!mma::wait(&empty[stage], phase ^ 1u, abort_flag, a.budget)) {
            report(a.status, kStTimeout, kWhereMuon + 2, t);
            ok = false;
            break;
          }
          // the next tile is drawn now: earlier, tiles would wait here that others could
          // begin with
          if (leader && kb == max(num_kb - kDrawAhead, 0)) mbar_arrive(near_end);
          const uint32_t bar = full0 + 8 * stage;
          if (leader) mbar_arrive_expect_tx(&full[stage], CG * 128 * (128 + G::kRowsB));
          mma::load_3d<CG>(s_a + stage * kOperand, ma, bar, (kb0 + kb) * 64, mrow, w.l);
          if (w.kind <= kPoly) mma::load_3d<CG>(s_b + stage * kOperand, mb, bar, (kb0 + kb) * 64, ncol, w.l);
          else mma::load_4d<CG>(s_b + stage * kOperand, mb, bar, 0, kb * 64, ncol >> 6, w.l);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {
        // loads on their way still land
        for (int i = 0; i < kStages; ++i) {
          const uint32_t par = i < stage ? phase : phase ^ 1u;
          const long long t0 = clock64();
          while (!mma::try_wait(&full[i], par) && clock64() - t0 < a.budget) {
          }
        }
      }
    }
  } else if (warp == G::kThreads / 32 - 1) {
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int slot = it % kRing;
      const uint32_t rph = (it / kRing) & 1;
      int t = -1;
      if (lane == 0) {
        if (leader) {
          ok = mma::wait(&rempty[slot], rph ^ 1u, abort_flag, a.budget) &&
               (it == 0 || mma::wait(near_end, (it - 1) & 1, abort_flag, a.budget));
          if (ok) {
            const int got = atomicAdd(a.counter, 1);
            t = got < total ? got : -1;
            ring[slot] = t;
            mbar_arrive(&rfull[slot]);
            if constexpr (CG == 2) mma::send_to_peer(&ring[slot], t, &rfull[slot]);
          }
        } else {
          ok = mma::wait(&rfull[slot], rph, abort_flag, a.budget);
          if (ok) {
            t = ring[slot];
            mma::arrive_at(rempty0 + 8 * slot);
          }
        }
        if (!ok) report(a.status, kStTimeout, kWhereMuon + 10, it);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      t = __shfl_sync(0xffffffffu, t, 0);
      if (!ok || t < 0) break;
      const Tile w = tile_of<kHalves>(t, a);
      const int num_kb = k_blocks(w, a);
      const int chunks = (num_kb + G::kChunk - 1) / G::kChunk;
      const int want = G::kDone * (w.kind == kGram ? w.step : w.step + 1);
      for (int c0 = 0; ok && c0 < chunks; c0 += 16) {
        // lanes 0 to 15 watch the first operand's counters, 16 to 31 the second one's
        const int mine = c0 + (lane & 15), most = min(chunks - c0, 16);
        const int* at = mine < chunks ? operand_counter(w, mine + w.part * (a.depth / G::kChunk), lane >> 4, a) : nullptr;
        bool ready = !at;
        int have = 0;                      // of these chunks, from the first on
        long long t0 = clock64();
        while (ok && have < most) {
          if (!ready) ready = acquire(at) >= want;
          const unsigned who = __ballot_sync(0xffffffffu, ready), both = who & who >> 16 & 0xffffu;
          const int now = min(most, __ffs(~both) - 1);
          if (now > have) {
            have = now;
            __threadfence_block();         // every lane's acquires before the word that tells of them
            __syncwarp();
            if (lane == 0) progress[slot] = operands_to(it, c0 + have);
            t0 = clock64();
          } else {
            const bool stop = *abort_flag || clock64() - t0 > a.budget;
            ok = !__any_sync(0xffffffffu, stop);
          }
        }
        if (!ok && lane == 0) {
          *abort_flag = 1;
          report(a.status, kStTimeout, kWhereMuon + 11, t);
        }
      }
      if (ok && lane == 0) mbar_arrive(&there[slot]);
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int slot = it % kRing;
        if (!mma::wait(&rfull[slot], (it / kRing) & 1, abort_flag, a.budget)) {
          report(a.status, kStTimeout, kWhereMuon + 3, it);
          break;
        }
        const int t = ring[slot];
        mbar_arrive(&rempty[slot]);
        if (t < 0) break;
        const Tile w = tile_of<kHalves>(t, a);
        const bool k_rows = w.kind > kPoly;        // X's rows are k
        const int num_kb = k_blocks(w, a);
        const uint32_t idesc = k_rows ? mma::idesc_f16_f32(G::kM, G::kN, false, true)
                                      : mma::idesc_f16_f32(G::kM, G::kN, false, false);
        const uint32_t b_lbo = k_rows ? 8192 : 16, b_step = k_rows ? 2048 : 32;
        const int buf = it & 1;
        if (!mma::wait(&tempty[buf], ((it >> 1) & 1) ^ 1u, abort_flag, a.budget)) {
          report(a.status, kStTimeout, kWhereMuon + 4, t);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * G::kN;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mma::wait(&full[stage], phase, abort_flag, a.budget)) {
            report(a.status, kStTimeout, kWhereMuon + 5, t);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(s_a + stage * kOperand), sb = smem_u32(s_b + stage * kOperand);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma::mma_f16<CG>(d, sdesc_sw128(sa + k * 32, 16, 1024), sdesc_sw128(sb + k * b_step, b_lbo, 1024), idesc,
                             kb > 0 || k > 0);
          mma::commit<CG>(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) mma::commit<CG>(&tfull[buf]);
      }
      mma::commit_here<CG>(drain);
      const long long t0 = clock64();
      while (!mma::try_wait(drain, 0) && clock64() - t0 < a.budget) {
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    constexpr int kCols = G::kN * 4 / G::kStore;
    Boxes b = {s_epi + (warp - 2) * kEpiWarp, &fetched[warp - 2], 0};
    const uint32_t tempty0 = mma::leader_addr<CG>(&tempty[0]);
    for (int it = 0;; ++it) {
      const int slot = it % kRing;
      const uint32_t rph = (it / kRing) & 1;
      if (!mma::warp_wait(&rfull[slot], rph, abort_flag, a.budget)) {
        report(a.status, kStTimeout, kWhereMuon + 6, it);
        break;
      }
      const int t = ring[slot];
      if (t >= 0 && !mma::warp_wait(&there[slot], rph, abort_flag, a.budget)) {
        report(a.status, kStTimeout, kWhereMuon + 7, t);
        break;
      }
      __syncwarp();
      if (lane == 0) mma::arrive_at(rempty0 + 8 * slot);
      if (t < 0) break;
      const Tile w = tile_of<kHalves>(t, a);
      const int buf = it & 1;
      const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * G::kN + half * kCols;
      const int row0 = w.m * G::kM + static_cast<int>(rank) * 128 + q * 32, n0 = w.n * G::kTile + w.half * G::kN + half * kCols;
      if (lane == 0 && row0 < a.n && n0 < (w.kind <= kPoly ? a.n : a.m)) {
        // the boxes are free: the tile before waited for its stores (and, Last, all
        // lanes are through with theirs)
        fence_async_global();
        if (w.kind == kPoly) fetch<kPoly>(a, w, b, row0, n0, 64);
        else if (w.kind >= kApply) fetch<kApply>(a, w, b, row0, n0, kCols);
      }
      if (!mma::warp_wait(&tfull[buf], (it >> 1) & 1, abort_flag, a.budget)) {
        report(a.status, kStTimeout, kWhereMuon + 8, t);
        break;
      }
      tc_fence_after();
      bool ok, mine = w.part == 0;
      const int slice = kHalves * (warp - 2) + w.half;
      if (w.kind == kGram) ok = epilogue<kGram, kCols>(a, w, tbase, row0, n0, lane, b, abort_flag, slice, mine);
      else if (w.kind == kPoly) ok = epilogue<kPoly, kCols>(a, w, tbase, row0, n0, lane, b, abort_flag, slice, mine);
      else if (w.kind == kApply) ok = epilogue<kApply, kCols>(a, w, tbase, row0, n0, lane, b, abort_flag, slice, mine);
      else ok = epilogue<kLast, kCols>(a, w, tbase, row0, n0, lane, b, abort_flag, slice, mine);
      if (!ok) {
        report(a.status, kStTimeout, kWhereMuon + 9, t);
        break;
      }
      tc_fence_before();
      if (w.kind == kLast) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mma::arrive_at(tempty0 + 8 * buf);
        if (w.kind != kLast && mine) {
          mma::stores_done();
          fence_async_global();
          const long long l = w.l;
          release_add(w.kind == kApply ? a.done_x + l * a.full + w.m * a.num_n + w.n
                                       : (w.kind == kGram ? a.done_a : a.done_b) + l * a.num_m * a.num_m +
                                             w.m * a.num_m + w.n);
        }
      }
    }
    if (lane == 0) mma::stores_done();
  }
  tc_fence_before();
  mma::sync_pair<CG>();
  if (warp == 1) {
    tc_fence_after();
    mma::tmem_free<CG, G::kCols>(tmem);
  }
}

// ------------------------------------------------------------- small matrices
//
// Up to 128 rows and 512 columns of X: a CTA does a matrix from its gradient to its
// update.  X's hi lies in shared memory as blocks of 64 columns, [128 rows][128 bytes],
// swizzled: the layout of an operand whose rows are the result's (X X^T) and, read the
// other way, of one whose rows are k (B X).  A and then B take two more such blocks, and lo
// as many as fit (16 KB a block of 64 columns too): all of them up to 384 columns, five of
// seven and four of eight beyond; the others' lo lies in the workspace, and comes from L2.
// No product waits for memory: 12 x [128][128] in fp32 take 78 us over the counters above,
// 24 here; 12 x [128][448] 55 and [128][512] 61 (53 and 59 with lo in eight
// bits, all of it in shared memory).

constexpr int kSmallRows = 128, kSmallCols = 512, kSmallThreads = 512;
constexpr int kBlock = 16384;
__host__ __device__ constexpr int small_blocks(int m) { return (m + 63) / 64; }
__host__ __device__ constexpr int small_lo(int blocks) { return blocks < 12 - blocks ? blocks : 12 - blocks; }
constexpr int small_bytes(int blocks) { return (blocks + small_lo(blocks) + 2) * kBlock + 1024 + 256; }
constexpr bool is_small(long long n, long long m) { return n <= kSmallRows && m <= kSmallCols; }

// Eight columns of row r in a block of lo, [8][128 rows] of eight values.
__device__ __forceinline__ uint4* small_lo_at(uint8_t* lo, int r, int j) {
  return reinterpret_cast<uint4*>(lo + (j * 128 + r) * 16);
}
// Eight columns (8 j0 on) of a row of X to their block of 64 and to lo's.
__device__ __forceinline__ void put_x(uint8_t* hi, uint8_t* lo, int r, int j0, const float (&v)[8]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = hi_bits(v[2 * j], v[2 * j + 1]);
    l[j] = lo_bits(v[2 * j], v[2 * j + 1], h[j]);
  }
  *swizzled(hi, r, j0) = make_uint4(h[0], h[1], h[2], h[3]);
  *small_lo_at(lo, r, j0) = make_uint4(l[0], l[1], l[2], l[3]);
}

template <typename G, typename M, bool kMom>
__global__ void __launch_bounds__(kSmallThreads) muon_small_kernel(const __grid_constant__ MuonArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* s_x = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                            ~static_cast<uintptr_t>(1023));
  const int blocks = small_blocks(a.m), near = small_lo(blocks);      // near: lo's in shared memory
  uint8_t* s_a = s_x + blocks * kBlock;
  uint8_t* s_lo = s_a + 2 * kBlock;
  uint64_t* bar = reinterpret_cast<uint64_t*>(s_lo + near * kBlock);
  uint32_t* slot = reinterpret_cast<uint32_t*>(bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);
  float* factor = reinterpret_cast<float*>(slot + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long l = blockIdx.x, base = l * a.rows * a.cols;
  const uint32_t cols = blocks <= 2 ? 128 : blocks <= 4 ? 256 : 512;
  uint8_t* far = a.far_lo + l * (blocks - near) * kBlock;
  auto lo_of = [&](int c) { return c < near ? s_lo + c * kBlock : far + (c - near) * kBlock; };
  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (l == 0) *a.status = DevStatus{0, 0, 0, 0};
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // the norm
  const G* grad = static_cast<const G*>(a.grad) + base;
  const M* mom = static_cast<const M*>(a.mom) + base;
  M* new_mom = static_cast<M*>(a.new_mom) + base;
  const int size = a.rows * a.cols;
  const bool flat = (size & 7) == 0 && aligned16(grad) && (!kMom || (aligned16(mom) && aligned16(new_mom)));
  const int count = flat ? size / 8 : size;
  double sum = 0.;
  auto add = [&](auto vec) {
    constexpr int VEC = decltype(vec)::value, kItems = VEC == 8 ? 2 : 8;
    for (int i0 = tid; i0 < count; i0 += kItems * kSmallThreads) {
      float g[kItems][VEC] = {};
      [[maybe_unused]] float m[kItems][VEC] = {};
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int i = i0 + k * kSmallThreads;
        if (i >= count) break;
        read_values(grad + VEC * i, g[k]);
        if constexpr (kMom) read_values(mom + VEC * i, m[k]);
      }
      if constexpr (kMom) updates_of(a, g, m);
      sum += squares(g);
    }
  };
  if (flat) add(std::integral_constant<int, 8>());
  else add(std::integral_constant<int, 1>());
  sum = block_sum<kSmallThreads>(sum);
  if (tid == 0) *factor = factor_of(sum, a.eps);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const float f = *factor;
  // X, zeros around it: eight columns of a row at a time, two times that on their way;
  // lanes next to one another along the rows of what came
  constexpr int kItems = 2;
  const bool vec = !a.tall && flat && (a.cols & 7) == 0;
  auto place = [&](int i, int& r, int& j0) {
    if (a.tall) {
      r = i % kSmallRows;
      j0 = i / kSmallRows;
    } else {
      const int eight = blocks * 8;
      r = i / eight;
      j0 = i - r * eight;
    }
  };
  auto source = [&](int r, int c) { return a.tall ? c * a.cols + r : r * a.cols + c; };
  const int items = kSmallRows * blocks * 8;         // a multiple of kItems * kSmallThreads
  for (int i0 = tid; i0 < items; i0 += kItems * kSmallThreads) {
    float v[kItems][8], m[kItems][8];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      int r, j0;
      place(i0 + k * kSmallThreads, r, j0);
      const int c = j0 * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = m[k][j] = 0.f;
      if (vec) {
        if (r < a.n && c < a.m) {
          read_values(grad + source(r, c), v[k]);
          if constexpr (kMom) read_values(mom + source(r, c), m[k]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r < a.n && c + j < a.m) {
            v[k][j] = to_f32(grad[source(r, c + j)]);
            if constexpr (kMom) m[k][j] = to_f32(mom[source(r, c + j)]);
          }
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      int r, j0;
      place(i0 + k * kSmallThreads, r, j0);
      const int c = j0 * 8;
      if constexpr (kMom) {
        float u[8];
        update_of<8>(a, v[k], m[k], u);
        if (vec) {
          if (r < a.n && c < a.m) write_values(new_mom + source(r, c), m[k]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float one[1] = {m[k][j]};
            if (r < a.n && c + j < a.m) store_vec<M, 1>(new_mom + source(r, c + j), one);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = u[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] *= f;
      put_x(s_x + (j0 >> 3) * kBlock, lo_of(j0 >> 3), r, j0 & 7, v[k]);
    }
  }

  const int q = warp & 3, quarter = warp >> 2, row = q * 32 + lane;
  const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
  uint32_t phase = 0;
  bool ok = true;
  // What the threads wrote is there for the tensor cores; then `issue` by one thread, and
  // everybody waits for its products.
  auto products = [&](auto issue) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      issue();
      mma::commit<1>(bar);
    }
    const bool done = mma::wait(bar, phase, abort_flag, a.budget);
    phase ^= 1u;
    ok = !__syncthreads_or(!done);
    tc_fence_after();
  };
  for (int step = 0; ok && step < a.steps; ++step) {
    const float ca = a.small_coeffs[3 * step], cb = a.small_coeffs[3 * step + 1], cc = a.small_coeffs[3 * step + 2];
    // A = X X^T
    products([&] {
      const uint32_t x = smem_u32(s_x);
      for (int k = 0; k < 4 * blocks; ++k) {
        const uint64_t d = sdesc_sw128(x + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024);
        mma::mma_f16<1>(tmem, d, d, mma::idesc_f16_f32(128, 128, false, false), k > 0);
      }
    });
    if (!ok) break;
    // this thread's 32 columns of A's row: half of a row of a block
    uint8_t* mine = s_a + (quarter >> 1) * 16384;
    const int j_a = (quarter & 1) * 4;
    float v[32];
    tmem_ld32(trow + quarter * 32, v);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *swizzled(mine, row, j_a + j) = make_uint4(
          hi_bits(v[8 * j] * kDown, v[8 * j + 1] * kDown), hi_bits(v[8 * j + 2] * kDown, v[8 * j + 3] * kDown),
          hi_bits(v[8 * j + 4] * kDown, v[8 * j + 5] * kDown), hi_bits(v[8 * j + 6] * kDown, v[8 * j + 7] * kDown));
    // B = a I + b A + c A A, in A's place
    products([&] {
      const uint32_t x = smem_u32(s_a);
      for (int k = 0; k < 8; ++k) {
        const uint64_t d = sdesc_sw128(x + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024);
        mma::mma_f16<1>(tmem, d, d, mma::idesc_f16_f32(128, 128, false, false), k > 0);
      }
    });
    if (!ok) break;
    tmem_ld32(trow + quarter * 32, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 r = *swizzled(mine, row, j_a + j);
      uint32_t h[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 x = hi_values(word_of(r, p));
        const int c = 8 * j + 2 * p;
        float b0 = fmaf(v[c], cc * kDown, cb * x.x), b1 = fmaf(v[c + 1], cc * kDown, cb * x.y);
        if (row == quarter * 32 + c) b0 += ca * kUp;
        if (row == quarter * 32 + c + 1) b1 += ca * kUp;
        h[p] = hi_bits(b0, b1);
      }
      *swizzled(mine, row, j_a + j) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    // X = B hi + a lo, up to 256 columns a product
    products([&] {
      const uint32_t x = smem_u32(s_x), b = smem_u32(s_a);
      for (int c = 0; c < blocks; c += 4) {
        const int w = min(blocks - c, 4);
        for (int k = 0; k < 8; ++k)
          mma::mma_f16<1>(tmem + 64 * c, sdesc_sw128(b + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024),
                          sdesc_sw128(x + c * 16384 + k * 2048, 16384, 1024),
                          mma::idesc_f16_f32(128, 64 * w, false, true), k > 0);
      }
    });
    if (!ok) break;
    const bool last = step + 1 == a.steps;
    const float fl = ca * kLoDown, up = a.scale * kDown;
    for (int u = quarter; u < 2 * blocks; u += 4) {
      tmem_ld32(trow + 32 * u, v);
      const int c = u >> 1;
      uint8_t* lo_c = lo_of(c);
      uint4 r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = *small_lo_at(lo_c, row, (u & 1) * 4 + i);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = (u & 1) * 4 + i;
        float x[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 lo = hi_values(word_of(r[i], p));
          x[2 * p] = fmaf(v[8 * i + 2 * p], kDown, fl * lo.x);
          x[2 * p + 1] = fmaf(v[8 * i + 2 * p + 1], kDown, fl * lo.y);
        }
        if (!last) {
          put_x(s_x + c * kBlock, lo_c, row, j, x);
        } else if (a.tall) {
#pragma unroll
          for (int p = 0; p < 8; ++p)
            if (row < a.n && c * 64 + 8 * j + p < a.m)
              a.out[base + source(row, c * 64 + 8 * j + p)] = __float2bfloat16_rn(x[p] * up);
        } else {
          *swizzled(s_x + c * 16384, row, j) =
              make_uint4(pack_bf16x2(x[0] * up, x[1] * up), pack_bf16x2(x[2] * up, x[3] * up),
                         pack_bf16x2(x[4] * up, x[5] * up), pack_bf16x2(x[6] * up, x[7] * up));
        }
      }
    }
  }
  if (ok && !a.tall) {
    // the update along its rows
    __syncthreads();
    const bool wide = (a.cols & 7) == 0 && aligned16(a.out + base);
    for (int i = tid; i < items; i += kSmallThreads) {
      int r, j0;
      place(i, r, j0);
      const int c = j0 * 8;
      if (r >= a.n || c >= a.m) continue;
      const uint4 w = *swizzled(s_x + (j0 >> 3) * 16384, r, j0 & 7);
      __nv_bfloat16* o = a.out + base + source(r, c);
      if (wide) {
        *reinterpret_cast<uint4*>(o) = w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t p = word_of(w, j / 2) >> (j % 2 * 16);
          if (c + j < a.m) reinterpret_cast<uint16_t*>(o)[j] = static_cast<uint16_t>(p);
        }
      }
    }
  }
  if (!ok && tid == 0) report(a.status, kStTimeout, kWhereMuon + 12, static_cast<int>(l));
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
  }
}

template <typename G, typename M, bool kMom>
cudaError_t run_small(const MuonArgs& args, cudaStream_t s) {
  static_assert(small_bytes(6) == small_bytes(small_blocks(kSmallCols)) && small_bytes(6) == small_bytes(7), "the most");
  const cudaError_t e = allow_smem<muon_small_kernel<G, M, kMom>>(small_bytes(6));
  if (e != cudaSuccess) return e;
  MuonArgs a = args;
  memcpy(a.small_coeffs, args.coeffs, sizeof(float) * 3 * static_cast<size_t>(a.steps));
  muon_small_kernel<G, M, kMom><<<static_cast<unsigned>(a.L), kSmallThreads, small_bytes(small_blocks(a.m)), s>>>(a);
  return cudaGetLastError();
}
template <typename G>
cudaError_t run_small(const MuonArgs& a, cudaStream_t s) {
  return !a.mom ? run_small<G, float, false>(a, s)
         : a.mom_bf16 ? run_small<G, __nv_bfloat16, true>(a, s) : run_small<G, float, true>(a, s);
}

// ------------------------------------------------------------------ the steps

bool map_of(MapEncoder enc, CUtensorMap* m, CUtensorMapDataType type, const void* base, int rank,
            const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [L][rows][cols] with row pitch ld, in boxes of bc columns x br rows.
bool map_3d(MapEncoder enc, CUtensorMap* m, const __half* base, long long cols, long long rows, long long L, long long ld,
            int bc, int br, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(L)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * 2 * rows};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(bc), static_cast<cuuint32_t>(br), 1};
  return map_of(enc, m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, 3, dims, strides, box, swizzle);
}

// The same as blocks of 64 columns, `blocks` of them x 64 rows a box: an operand whose rows
// are k.  Columns past `cols` in the last block come from the rows' padding; they
// reach only results past the result's last column.
bool map_k_rows(MapEncoder enc, CUtensorMap* m, const __half* base, long long cols, long long rows, long long L,
                long long ld, int blocks) {
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>((cols + 63) / 64),
                              static_cast<cuuint64_t>(L)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld) * 2, 128, static_cast<cuuint64_t>(ld) * 2 * rows};
  const cuuint32_t box[4] = {64, 64, static_cast<cuuint32_t>(blocks), 1};
  return map_of(enc, m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int CG, int kHalves>
cudaError_t run_steps(const MuonArgs& a, MapEncoder enc, int num_sms, cudaStream_t s) {
  using G = Geo<CG, kHalves>;
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    ok = ok && map_3d(enc, &g.xk[i], a.x[i].hi, a.m, a.n, a.L, a.ldx, 64, 128) &&
         map_3d(enc, &g.xs[i], a.x[i].hi, a.m, a.n, a.L, a.ldx, 64, G::kRowsB) &&
         map_k_rows(enc, &g.xn[i], a.x[i].hi, a.m, a.n, a.L, a.ldx, G::kRowsB / 64) &&
         map_3d(enc, &g.xh[i], a.x[i].hi, a.m, a.n, a.L, a.ldx, 64, 32) &&
         map_3d(enc, &g.xl[i], a.x[i].lo, a.m, a.n, a.L, a.ldx, 64, 32);
  }
  ok = ok && map_3d(enc, &g.ak, a.gram, a.n, a.n, a.L, a.lda, 64, 128) &&
       map_3d(enc, &g.a2, a.gram, a.n, a.n, a.L, a.lda, 64, G::kRowsB) &&
       map_3d(enc, &g.as, a.gram, a.n, a.n, a.L, a.lda, 64, 32) &&
       map_3d(enc, &g.at, a.gram, a.n, a.n, a.L, a.lda, 32, 64, CU_TENSOR_MAP_SWIZZLE_NONE) &&
       map_3d(enc, &g.bk, a.poly, a.n, a.n, a.L, a.lda, 64, 128) &&
       map_3d(enc, &g.bs, a.poly, a.n, a.n, a.L, a.lda, 64, 32) &&
       map_3d(enc, &g.bt, a.poly, a.n, a.n, a.L, a.lda, 32, 64, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (!ok) return cudaErrorInvalidValue;
  constexpr int T = G::kTile;
  g.n = a.n;
  g.m = a.m;
  g.L = a.L;
  g.steps = a.steps;
  g.num_m = (a.n + T - 1) / T;
  g.num_n = (a.m + T - 1) / T;
  g.tri = g.num_m * (g.num_m + 1) / 2;
  g.full = g.num_m * g.num_n;
  g.depth = (g.m + 63) / 64;
  g.split = 1;
  if (CG == 1 && a.split > 1) {
    g.depth = ((g.depth + a.split - 1) / a.split + G::kChunk - 1) / G::kChunk * G::kChunk;
    g.split = ((g.m + 63) / 64 + g.depth - 1) / g.depth;
  }
  g.parts = a.parts;
  memcpy(g.coeffs, a.coeffs, sizeof(float) * 3 * static_cast<size_t>(a.steps));
  g.out = a.out;
  g.scale = a.scale;
  g.tall = a.tall;
  g.counter = a.sync;
  g.done_a = a.sync + 32;
  g.done_b = g.done_a + static_cast<long long>(a.L) * g.num_m * g.num_m;
  g.done_x = g.done_b + static_cast<long long>(a.L) * g.num_m * g.num_m;
  g.arrived = g.done_x + static_cast<long long>(a.L) * g.full;
  g.status = a.status;
  g.budget = a.budget;
  const auto kernel = muon_gemm_kernel<CG, kHalves>;
  cudaError_t e = allow_smem<muon_gemm_kernel<CG, kHalves>>(kSmem);
  if (e != cudaSuccess) return e;
  // a CTA an SM at most; CTAs wait for one another, so they are launched to run
  // together
  const long long tiles = static_cast<long long>(g.tri * g.split + g.tri + g.full) * a.L * a.steps * kHalves, most = num_sms / CG;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {CG, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(CG * (tiles < most ? tiles : most)));
  cfg.blockDim = dim3(G::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kernel, g);
}

template <typename G, typename M, bool kMom>
cudaError_t prepare(const MuonArgs& a, int num_sms, cudaStream_t s) {
  const dim3 chunks(static_cast<unsigned>(a.chunks), static_cast<unsigned>(a.L));
  muon_norm_kernel<G, M, kMom><<<chunks, kPrepThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>((a.m + 63) / 64) * ((a.n + 63) / 64), most = 8LL * num_sms;
  const dim3 grid(static_cast<unsigned>(tiles < most ? tiles : most), static_cast<unsigned>(a.L));
  return a.tall ? launch_overlapped(muon_scale_kernel<G, M, kMom, true>, grid, dim3(kPrepThreads), 0, s, a)
                : launch_overlapped(muon_scale_kernel<G, M, kMom, false>, grid, dim3(kPrepThreads), 0, s, a);
}
template <typename G>
cudaError_t prepare(const MuonArgs& a, int num_sms, cudaStream_t s) {
  return !a.mom ? prepare<G, float, false>(a, num_sms, s)
         : a.mom_bf16 ? prepare<G, __nv_bfloat16, true>(a, num_sms, s) : prepare<G, float, true>(a, num_sms, s);
}

}  // namespace

// Parts of a tile of A along k (where tiles are 128 x 128 or halves of that): a few long
// products would leave most SMs idle.  A part of k-blocks takes 416 to 555 clocks each, a
// part's sum 64 KB from L2, twice that: ten k-blocks a part at least, eight parts at most,
// and all of them at once as halves on a GB300's 152 SMs ([640][8192] 220 us, 228 with four
// parts instead of five).  It goes by that number and not by the device's, since it decides
// the workspace's size, which is asked for without a device; with fewer SMs the parts
// take turns.  [129][8000] 131 us, 249 in one part; [200][3000] 109 and 139.
constexpr long long kSplitTiles = 152 / 2;
static long long gram_split(long long L, long long n, long long m) {
  const long long tn = (n + 127) / 128, tri = tn * (tn + 1) / 2, kb = (m + 63) / 64;
  const long long most = L > 0 ? kSplitTiles / (L * tri) : 0, s = kb / 10 < most ? kb / 10 : most;
  return s > 8 ? 8 : s < 1 ? 1 : s;
}

MuonPlan muon_plan(long long L, long long rows, long long cols) {
  MuonPlan p = {};
  const long long n = rows < cols ? rows : cols, m = rows < cols ? cols : rows, size = n * m;
  auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  if (is_small(n, m)) {
    const int blocks = small_blocks(static_cast<int>(m));
    p.far_lo = up(sizeof(DevStatus));
    p.total = p.far_lo + static_cast<size_t>(L * (blocks - small_lo(blocks)) * kBlock);
    return p;
  }
  p.ldx = (m + 63) / 64 * 64;
  p.lda = (n + 63) / 64 * 64;
  p.chunk = (size + kMostChunks - 1) / kMostChunks;
  if (p.chunk < kChunk) p.chunk = kChunk;
  p.chunk = (p.chunk + 7) / 8 * 8;
  p.chunks = (size + p.chunk - 1) / p.chunk;
  const size_t x = up(static_cast<size_t>(2 * L * n * p.ldx)), q = up(static_cast<size_t>(2 * L * n * p.lda));
  // a drawing counter (a line of its own) and one a tile, of the smaller tiles
  const size_t tn = static_cast<size_t>((n + 127) / 128), tm = static_cast<size_t>((m + 127) / 128);
  p.split = gram_split(L, n, m);
  const size_t slices = static_cast<size_t>(L) * (tn * (tn + 1) / 2) * kStoreWarps;
  p.sync_words = 32 + static_cast<size_t>(L) * tn * (2 * tn + tm) + slices;
  p.sync = up(sizeof(DevStatus));
  p.partial = p.sync + up(4 * p.sync_words);
  p.x[0] = p.partial + up(static_cast<size_t>(8 * L * p.chunks));
  for (int i = 1; i < 4; ++i) p.x[i] = p.x[i - 1] + x;
  p.gram = p.x[3] + x;
  p.poly = p.gram + q;
  p.parts = p.poly + q;
  p.total = p.parts + (p.split > 1 ? slices * static_cast<size_t>(p.split) * 8192 : 0);
  return p;
}

cudaError_t launch_muon(const MuonArgs& a, int grad_bf16, MapEncoder enc, int num_sms, cudaStream_t s) {
  if (is_small(a.n, a.m)) return grad_bf16 ? run_small<__nv_bfloat16>(a, s) : run_small<float>(a, s);
  const cudaError_t e = grad_bf16 ? prepare<__nv_bfloat16>(a, num_sms, s) : prepare<float>(a, num_sms, s);
  if (e != cudaSuccess) return e;
  // Products are deep (n or m) and few tiles wide where matrices are small, so the rule
  // goes by X's tiles of 128 x 128.  Where each SM gets half of one at most, halves, which
  // take in 24 KB a k-block instead of 32 ([1003][777] 128 us and 139, [320][320] 81 and
  // 95).  Where it gets few, whole ones, X X^T of few tiles in parts ([2048][2048] 258 us
  // and 274 by pairs, [640][8192] 221 and 336).  Else 256 x 256 tiles by pairs, which take
  // in half the bytes an operation ([2560][2560], 2.6 tiles an SM, 349 us and 401).  That
  // matters less the less deep the products are (2 x [384][4096], 152 us and 207;
  // 3 x [300][8000], 3.7 an SM, 220 and 331; 8 x [320][4096], 5 an SM, 274 and 273), and
  // at 128 rows or fewer pairs would be half empty (12 x [128][4096] 157 us and 234).
  const long long small = static_cast<long long>(a.L) * ((a.n + 127) / 128) * ((a.m + 127) / 128);
  const bool single = a.n <= 128 || 4 * small <= (a.n <= 384 ? 16LL : 9LL) * num_sms;
  return !single               ? run_steps<2, 1>(a, enc, num_sms, s)
         : 2 * small > num_sms ? run_steps<1, 1>(a, enc, num_sms, s)
                               : run_steps<1, 2>(a, enc, num_sms, s);
}

}  // namespace eas
