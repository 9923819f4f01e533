// Orthogonalised update of a matrix: momentum, then Newton-Schulz products.
//
//   m' = beta m + (1 - beta) g,  u = m' or (1 - beta) g + beta m',
//   X = u / (|u| + eps), transposed where it is taller than wide: [n][m], n <= m;
//   each step  A = X X^T,  B = b A + c A A,  X = a X + B X;  out = scale X.
//
// The products run on the tensor cores with fp16 operands and fp32 accumulators.
// X is kept as a pair of fp16, hi + lo (22 bits); only hi is multiplied, and a X takes
// both.  What decides the precision is X's own rounding: an error in a direction of
// small singular values grows with them by a each step, beside large ones that do
// not grow.  On gradients of low rank with noise, X in one fp16 ends 5e-3 off, in bf16
// 4e-2, as a pair 2e-4 (512 to 1024 rows, five steps; the output's rounding to bf16 is
// 1.7e-3).  The roundings of A, B and of hi in the products stay where they are, each
// step's 2^-11 of its own product.  Everything is stored times 2^12, so that fp16's range covers
// entries from 2^-36 to 16.
//
// A and A A are symmetric: only tiles on and above the diagonal are computed, and
// stored twice, the second time transposed.  A step takes 3 n^2 m + n^3 operations.
#include <cstring>

#include <cuda_fp16.h>

#include "eas_launch.cuh"
#include "eas_mma.cuh"
#include "eas_ops.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr float kUp = 4096.f, kDown = 1.f / 4096.f;   // the stored scale
constexpr int kWhereMuon = 50;

// ------------------------------------------------- momentum, norm, conversion

constexpr int kPrepThreads = 256;
constexpr int kChunk = 16384;     // elements a CTA at least
constexpr int kMostChunks = 1024; // partial sums a matrix

template <typename T>
__device__ __forceinline__ float load1(const void* p, long long i) {
  return to_f32(static_cast<const T*>(p)[i]);
}

// Sum of squares in fp64, added up in fp32 over a vector where that is safe.
template <int VEC>
__device__ __forceinline__ double squares(const float (&u)[VEC]) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < VEC; ++j) s = fmaf(u[j], u[j], s);
  if (s > 1e-30f && s < 1e30f) return s;
  double d = 0.;
#pragma unroll
  for (int j = 0; j < VEC; ++j) d += static_cast<double>(u[j]) * u[j];
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

// Each CTA a chunk of a matrix: the new momentum, u (fp32) where there is a momentum,
// and the chunk's sum of squares.
template <typename G, typename M, bool kMom, bool kVec>
__device__ double update_chunk(const MuonArgs& a, long long base, long long lo, long long hi) {
  constexpr int VEC = kVec ? 8 : 1;
  const float beta = a.beta, rest = a.rest;
  double sum = 0.;
  for (long long i = lo + static_cast<long long>(threadIdx.x) * VEC; i < hi; i += kPrepThreads * VEC) {
    float g[VEC], u[VEC];
    read_values(static_cast<const G*>(a.grad) + base + i, g);
    if constexpr (kMom) {
      float m[VEC];
      read_values(static_cast<const M*>(a.mom) + base + i, m);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        m[j] = fmaf(beta, m[j], rest * g[j]);
        u[j] = a.nesterov ? fmaf(beta, m[j], rest * g[j]) : m[j];
      }
      write_values(static_cast<M*>(a.new_mom) + base + i, m);
      write_values(a.u + base + i, u);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) u[j] = g[j];
    }
    sum += squares<VEC>(u);
  }
  return sum;
}

// Sum over the CTA, in thread 0.
__device__ double block_sum(double v) {
  __shared__ double part[kPrepThreads / 32];
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_down_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.;
    for (int w = 0; w < kPrepThreads / 32; ++w) v += part[w];
  }
  return v;
}

// grid (chunks, L)
template <typename G, typename M, bool kMom>
__global__ void __launch_bounds__(kPrepThreads) muon_update_kernel(const MuonArgs a) {
  const long long size = static_cast<long long>(a.rows) * a.cols, base = blockIdx.y * size;
  const long long lo = blockIdx.x * a.chunk, hi = lo + a.chunk < size ? lo + a.chunk : size;
  bool vec = (size & 7) == 0 && aligned16(a.grad);
  if constexpr (kMom) vec = vec && aligned16(a.mom) && aligned16(a.new_mom);
  const double sum = block_sum(vec ? update_chunk<G, M, kMom, true>(a, base, lo, hi)
                                   : update_chunk<G, M, kMom, false>(a, base, lo, hi));
  if (threadIdx.x == 0) {
    a.partial[blockIdx.y * gridDim.x + blockIdx.x] = sum;
    if (blockIdx.x == 0 && blockIdx.y == 0) *a.status = DevStatus{0, 0, 0, 0};
  }
}

// X's first pair: u (or the gradient) times 2^12 / (norm + eps), transposed where it
// is taller than wide.  A CTA a 64 x 64 tile; grid (tiles of X's columns, of its
// rows, L).
template <typename G>
__global__ void __launch_bounds__(kPrepThreads) muon_scale_kernel(const MuonArgs a) {
  __shared__ float tile[64][65];
  __shared__ float factor;
  const int tid = threadIdx.x, l = blockIdx.z;
  wait_for_launch_before();
  double s = 0.;
  for (int i = tid; i < a.chunks; i += kPrepThreads) s += a.partial[static_cast<long long>(l) * a.chunks + i];
  s = block_sum(s);
  if (tid == 0) factor = static_cast<float>(kUp / (sqrt(s) + a.eps));
  const long long base = static_cast<long long>(l) * a.rows * a.cols;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;        // of X
  auto value = [&](int r, int c) {
    const long long i = base + static_cast<long long>(r) * a.cols + c;
    return a.mom ? a.u[i] : load1<G>(a.grad, i);
  };
  if (a.tall) {
    for (int i = tid; i < 64 * 64; i += kPrepThreads) {
      const int c = i / 64, r = i % 64;                        // consecutive r: consecutive in memory
      tile[r][c] = r0 + r < a.n && c0 + c < a.m ? value(c0 + c, r0 + r) : 0.f;
    }
  }
  __syncthreads();
  const float f = factor;
  for (int i = tid; i < 64 * 32; i += kPrepThreads) {
    const int r = i / 32, c = i % 32 * 2;
    if (r0 + r >= a.n) break;
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (a.tall) v[j] = tile[r][c + j];
      else v[j] = c0 + c + j < a.m ? value(r0 + r, c0 + c + j) : 0.f;
      v[j] *= f;
    }
    const __half2 hi = __floats2half2_rn(v[0], v[1]);
    const __half2 lo = __floats2half2_rn(v[0] - __low2float(hi), v[1] - __high2float(hi));
    const long long o = (static_cast<long long>(l) * a.n + r0 + r) * a.ldx + c0 + c;
    *reinterpret_cast<__half2*>(a.x[0].hi + o) = hi;
    *reinterpret_cast<__half2*>(a.x[0].lo + o) = lo;
  }
}

// ------------------------------------------------------------------ products

enum Kind { kGram, kPoly, kApply, kLast };

constexpr int kThreads = 192;
constexpr int kStages = 6;
constexpr int kOperand = 16384;                    // 128 rows (columns) x 64 k
constexpr int kEpiWarp = 8192;                     // two boxes a warp
constexpr int kSmem = kStages * 2 * kOperand + 4 * kEpiWarp + 1024 + 512;

// CG = 2: a pair of CTAs computes 256 x 256 tiles, each 128 of the rows; CG = 1: a CTA
// 128 x 128 tiles.
template <int CG>
struct Geo {
  static constexpr int kM = 128 * CG, kN = 128 * CG;
  static constexpr uint32_t kCols = 2 * kN;        // two accumulators
};

struct GemmArgs {
  CUtensorMap ma, mb;       // operands
  CUtensorMap s0, s1;       // stores: the tile; its transpose (Gram, Poly) or lo (Apply)
  int n, m, L;              // extents of the result: n x n (Gram, Poly) or n x m
  int num_kb;               // 64-deep k-blocks
  int num_m, num_n, per;    // tiles a matrix
  float ca, cb, cc;         // the step's coefficients
  const __half* p0;         // Poly: A; Apply, Last: X hi
  const __half* p1;         // Apply, Last: X lo
  long long ld;             // their row pitch
  __nv_bfloat16* out;       // Last
  float scale;
  int tall;
  DevStatus* status;
  long long budget;
};

struct Tile {
  int l, m, n;
};

template <int kKind>
__device__ __forceinline__ Tile tile_of(int t, const GemmArgs& a) {
  Tile w;
  w.l = t / a.per;
  t -= w.l * a.per;
  if constexpr (kKind <= kPoly) {
    // column by column of the upper triangle: n (n + 1) / 2 tiles before column n
    int n = static_cast<int>((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
    while (n * (n + 1) / 2 > t) --n;
    while ((n + 1) * (n + 2) / 2 <= t) ++n;
    w.n = n;
    w.m = t - n * (n + 1) / 2;
  } else {
    // the tiles of one column strip of X together: they share its k-blocks
    w.n = t / a.num_m;
    w.m = t - w.n * a.num_m;
  }
  return w;
}

// 64 columns of this thread's accumulator row.
__device__ __forceinline__ void load64(uint32_t taddr, float (&v)[64]) {
  tmem_ld32(taddr, *reinterpret_cast<float(*)[32]>(&v[0]));
  tmem_ld32(taddr + 32, *reinterpret_cast<float(*)[32]>(&v[32]));
}

// 64 fp16 values of a row in global memory.
__device__ __forceinline__ void row64(const __half* p, uint4 (&r)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = reinterpret_cast<const uint4*>(p)[j];
}
__device__ __forceinline__ float2 pair_of(const uint4 (&r)[8], int i) {
  const uint32_t w[4] = {r[i / 4].x, r[i / 4].y, r[i / 4].z, r[i / 4].w};
  return __half22float2(*reinterpret_cast<const __half2*>(&w[i % 4]));
}

// The row of a [32][64] fp16 box in the 128-byte swizzled layout: value pair i.
__device__ __forceinline__ void put_box(uint8_t* box, int lane, const uint32_t (&w)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One warp's 32 rows (from row0 on; this thread's is row0 + lane) of a tile whose
// first column is n0.
template <int kKind, int kTileN>
__device__ __forceinline__ void epilogue(const GemmArgs& a, const Tile& w, uint32_t tbase, int row0, int n0,
                                         int lane, uint8_t* box) {
  const int width = kKind <= kPoly ? a.n : a.m;
  const int row = row0 + lane;
  const bool mirror = kKind <= kPoly && w.m != w.n;
#pragma unroll 1
  for (int c = 0; c < kTileN / 64; ++c) {
    const int col = n0 + c * 64;
    if (col >= width || row0 >= a.n) break;        // the same for the warp
    float v[64];
    load64(tbase + c * 64, v);
    if constexpr (kKind == kGram) {
#pragma unroll
      for (int j = 0; j < 64; ++j) v[j] *= kDown;
    } else {
      // rows past the end read the last one; they are not stored
      const long long o = (static_cast<long long>(w.l) * a.n + min(row, a.n - 1)) * a.ld + col;
      uint4 r[8];
      row64(a.p0 + o, r);
      const float f = kKind == kPoly ? a.cb : a.ca, g = kKind == kPoly ? a.cc * kDown : kDown;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 x = pair_of(r, j);
        v[2 * j] = fmaf(v[2 * j], g, f * x.x);
        v[2 * j + 1] = fmaf(v[2 * j + 1], g, f * x.y);
      }
      if constexpr (kKind >= kApply) {
        row64(a.p1 + o, r);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float2 x = pair_of(r, j);
          v[2 * j] = fmaf(f, x.x, v[2 * j]);
          v[2 * j + 1] = fmaf(f, x.y, v[2 * j + 1]);
        }
      }
    }
    if constexpr (kKind == kLast) {
      const float f = a.scale * kDown;
      if (a.tall) {
        // X's rows are the output's columns: 32 lanes store 64 bytes in a row
        if (row < a.n) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (col + j < a.m)
              a.out[(static_cast<long long>(w.l) * a.m + col + j) * a.n + row] = __float2bfloat16_rn(v[j] * f);
        }
      } else {
        uint32_t* s = reinterpret_cast<uint32_t*>(box);      // [32][33] pairs
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) s[lane * 33 + j] = pack_bf16x2(v[2 * j] * f, v[2 * j + 1] * f);
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
      uint32_t hi[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) hi[j] = half2_bits(v[2 * j], v[2 * j + 1]);
      if (lane == 0) mma::stores_read();             // the boxes' last stores have read them
      __syncwarp();
      put_box(box, lane, hi);
      if constexpr (kKind == kApply) {
        uint32_t lo[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
          lo[j] = half2_bits(v[2 * j] - h.x, v[2 * j + 1] - h.y);
        }
        put_box(box + 4096, lane, lo);
      } else if (mirror) {
        // [64][32]: the columns as rows
        __half* t = reinterpret_cast<__half*>(box + 4096);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const __half2 h = *reinterpret_cast<const __half2*>(&hi[j]);
          t[(2 * j) * 32 + lane] = __low2half(h);
          t[(2 * j + 1) * 32 + lane] = __high2half(h);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mma::store_3d(&a.s0, box, col, row0, w.l);
        if constexpr (kKind == kApply) mma::store_3d(&a.s1, box + 4096, col, row0, w.l);
        else if (mirror) mma::store_3d(&a.s1, box + 4096, row0, col, w.l);
        mma::store_commit();
      }
    }
  }
}

// Persistent: CTA (pair) p computes tiles p, p + grid, ...  Warp 0 loads, warp 1
// issues the MMAs, warps 2 to 5 store; two accumulators, so that a tile's store runs
// under the next one's products.
template <int CG, int kKind>
__global__ void __launch_bounds__(kThreads, 1) muon_gemm_kernel(const __grid_constant__ GemmArgs a) {
  using G = Geo<CG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* s_a = smem;
  uint8_t* s_b = smem + kStages * kOperand;
  uint8_t* s_epi = s_b + kStages * kOperand;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_epi + 4 * kEpiWarp);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);

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
      mbar_init(&tempty[i], 4 * CG);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&a.ma);
    tma_prefetch_desc(&a.mb);
  }
  if (warp == 1) mma::tmem_alloc<CG, G::kCols>(slot);
  tc_fence_before();
  mma::sync_pair<CG>();
  tc_fence_after();
  const uint32_t tmem = *slot;
  // the set-up above overlaps the launch before; nothing of its output is read
  // earlier
  wait_for_launch_before();
  launch_dependents();

  const int total = a.per * a.L, step = gridDim.x / CG, first = blockIdx.x / CG;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t full0 = mma::leader_addr<CG>(&full[0]);
      for (int t = first; ok && t < total; t += step) {
        const Tile w = tile_of<kKind>(t, a);
        const int mrow = w.m * G::kM + static_cast<int>(rank) * 128;
        const int ncol = w.n * G::kN + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < a.num_kb; ++kb) {
          if (!mma::wait(&empty[stage], phase ^ 1u, abort_flag, a.budget)) {
            report(a.status, kStTimeout, kWhereMuon, t);
            ok = false;
            break;
          }
          const uint32_t bar = full0 + 8 * stage;
          if (leader) mbar_arrive_expect_tx(&full[stage], CG * 2 * kOperand);
          mma::load_3d<CG>(s_a + stage * kOperand, &a.ma, bar, kb * 64, mrow, w.l);
          if constexpr (kKind <= kPoly)
            mma::load_3d<CG>(s_b + stage * kOperand, &a.mb, bar, kb * 64, ncol, w.l);
          else
            mma::load_4d<CG>(s_b + stage * kOperand, &a.mb, bar, 0, kb * 64, ncol >> 6, w.l);
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
  } else if (warp == 1) {
    if (leader && lane == 0) {
      constexpr uint32_t idesc = mma::idesc_f16_f32(G::kM, G::kN, false, kKind > kPoly);
      constexpr uint32_t b_lbo = kKind > kPoly ? 8192 : 16, b_step = kKind > kPoly ? 2048 : 32;
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; ok && t < total; t += step, ++it) {
        const int buf = it & 1;
        if (!mma::wait(&tempty[buf], ((it >> 1) & 1) ^ 1u, abort_flag, a.budget)) {
          report(a.status, kStTimeout, kWhereMuon + 1, t);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * G::kN;
        for (int kb = 0; kb < a.num_kb; ++kb) {
          if (!mma::wait(&full[stage], phase, abort_flag, a.budget)) {
            report(a.status, kStTimeout, kWhereMuon + 2, t);
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
    const int q = warp & 3;
    uint8_t* box = s_epi + q * kEpiWarp;
    const uint32_t tempty0 = mma::leader_addr<CG>(&tempty[0]);
    int it = 0;
    for (int t = first; t < total; t += step, ++it) {
      const Tile w = tile_of<kKind>(t, a);
      const int buf = it & 1;
      if (!mma::wait(&tfull[buf], (it >> 1) & 1, abort_flag, a.budget)) {
        report(a.status, kStTimeout, kWhereMuon + 3, t);
        break;
      }
      tc_fence_after();
      epilogue<kKind, G::kN>(a, w, tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * G::kN,
                             w.m * G::kM + static_cast<int>(rank) * 128 + q * 32, w.n * G::kN, lane, box);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mma::arrive_at(tempty0 + 8 * buf);
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

template <int CG, int kKind>
cudaError_t launch_gemm(const GemmArgs& a, int num_sms, cudaStream_t s) {
  cudaError_t e = allow_smem<muon_gemm_kernel<CG, kKind>>(kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>(a.per) * a.L, most = num_sms / CG;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {CG, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(CG * (tiles < most ? tiles : most)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, muon_gemm_kernel<CG, kKind>, a);
}

// ------------------------------------------------------------------ the steps

bool map_of(MapEncoder enc, CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, bool swizzled) {
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides,
             box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [L][rows][cols] with row pitch ld, in boxes of bc columns x br rows.
bool map_3d(MapEncoder enc, CUtensorMap* m, const __half* base, long long cols, long long rows, long long L,
            long long ld, int bc, int br, bool swizzled = true) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(L)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * 2 * rows};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(bc), static_cast<cuuint32_t>(br), 1};
  return map_of(enc, m, base, 3, dims, strides, box, swizzled);
}

// The same as blocks of 64 columns, two blocks x 64 rows a box: an operand whose rows
// are k.  Columns past `cols` in the last block come from the rows' padding; they
// reach only results past the result's last column.
bool map_k_rows(MapEncoder enc, CUtensorMap* m, const __half* base, long long cols, long long rows, long long L,
                long long ld) {
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>((cols + 63) / 64),
                              static_cast<cuuint64_t>(L)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(ld) * 2, 128, static_cast<cuuint64_t>(ld) * 2 * rows};
  const cuuint32_t box[4] = {64, 64, 2, 1};
  return map_of(enc, m, base, 4, dims, strides, box, true);
}

template <int CG>
cudaError_t run_steps(const MuonArgs& a, MapEncoder enc, int num_sms, cudaStream_t s) {
  constexpr int T = 128 * CG;
  CUtensorMap xk[2], xn[2], xh[2], xl[2], ak, as, at, bk, bs, bt;
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    ok = ok && map_3d(enc, &xk[i], a.x[i].hi, a.m, a.n, a.L, a.ldx, 64, 128);
    ok = ok && map_k_rows(enc, &xn[i], a.x[i].hi, a.m, a.n, a.L, a.ldx);
    ok = ok && map_3d(enc, &xh[i], a.x[i].hi, a.m, a.n, a.L, a.ldx, 64, 32);
    ok = ok && map_3d(enc, &xl[i], a.x[i].lo, a.m, a.n, a.L, a.ldx, 64, 32);
  }
  ok = ok && map_3d(enc, &ak, a.gram, a.n, a.n, a.L, a.lda, 64, 128) &&
       map_3d(enc, &as, a.gram, a.n, a.n, a.L, a.lda, 64, 32) &&
       map_3d(enc, &at, a.gram, a.n, a.n, a.L, a.lda, 32, 64, false) &&
       map_3d(enc, &bk, a.poly, a.n, a.n, a.L, a.lda, 64, 128) &&
       map_3d(enc, &bs, a.poly, a.n, a.n, a.L, a.lda, 64, 32) &&
       map_3d(enc, &bt, a.poly, a.n, a.n, a.L, a.lda, 32, 64, false);
  if (!ok) return cudaErrorInvalidValue;
  GemmArgs g;
  memset(&g, 0, sizeof(g));
  g.n = a.n;
  g.m = a.m;
  g.L = a.L;
  g.num_m = (a.n + T - 1) / T;
  g.out = a.out;
  g.scale = a.scale;
  g.tall = a.tall;
  g.status = a.status;
  g.budget = a.budget;
  for (int i = 0; i < a.steps; ++i) {
    const MuonPair &x = a.x[i & 1];
    const int to = (i + 1) & 1;
    g.ca = a.coeffs[3 * i];
    g.cb = a.coeffs[3 * i + 1];
    g.cc = a.coeffs[3 * i + 2];
    // A = X X^T
    g.ma = g.mb = xk[i & 1];
    g.s0 = as;
    g.s1 = at;
    g.num_kb = (a.m + 63) / 64;
    g.num_n = g.num_m;
    g.per = g.num_m * (g.num_m + 1) / 2;
    cudaError_t e = launch_gemm<CG, kGram>(g, num_sms, s);
    if (e != cudaSuccess) return e;
    // B = b A + c A A
    g.ma = g.mb = ak;
    g.s0 = bs;
    g.s1 = bt;
    g.num_kb = (a.n + 63) / 64;
    g.p0 = a.gram;
    g.ld = a.lda;
    e = launch_gemm<CG, kPoly>(g, num_sms, s);
    if (e != cudaSuccess) return e;
    // X = a X + B X
    g.ma = bk;
    g.mb = xn[i & 1];
    g.s0 = xh[to];
    g.s1 = xl[to];
    g.num_n = (a.m + T - 1) / T;
    g.per = g.num_m * g.num_n;
    g.p0 = x.hi;
    g.p1 = x.lo;
    g.ld = a.ldx;
    e = i + 1 < a.steps ? launch_gemm<CG, kApply>(g, num_sms, s) : launch_gemm<CG, kLast>(g, num_sms, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename G>
cudaError_t prepare(const MuonArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.chunks), static_cast<unsigned>(a.L));
  if (!a.mom) muon_update_kernel<G, float, false><<<grid, kPrepThreads, 0, s>>>(a);
  else if (a.mom_bf16) muon_update_kernel<G, __nv_bfloat16, true><<<grid, kPrepThreads, 0, s>>>(a);
  else muon_update_kernel<G, float, true><<<grid, kPrepThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 tiles(static_cast<unsigned>((a.m + 63) / 64), static_cast<unsigned>((a.n + 63) / 64),
                   static_cast<unsigned>(a.L));
  return launch_overlapped(muon_scale_kernel<G>, tiles, dim3(kPrepThreads), 0, s, a);
}

}  // namespace

MuonPlan muon_plan(long long L, long long rows, long long cols) {
  MuonPlan p;
  const long long n = rows < cols ? rows : cols, m = rows < cols ? cols : rows, size = n * m;
  p.ldx = (m + 63) / 64 * 64;
  p.lda = (n + 63) / 64 * 64;
  p.chunk = (size + kMostChunks - 1) / kMostChunks;
  if (p.chunk < kChunk) p.chunk = kChunk;
  p.chunk = (p.chunk + 7) / 8 * 8;
  p.chunks = (size + p.chunk - 1) / p.chunk;
  auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  const size_t x = up(static_cast<size_t>(2 * L * n * p.ldx)), q = up(static_cast<size_t>(2 * L * n * p.lda));
  p.partial = up(sizeof(DevStatus));
  p.x[0] = p.partial + up(static_cast<size_t>(8 * L * p.chunks));
  for (int i = 1; i < 4; ++i) p.x[i] = p.x[i - 1] + x;
  p.gram = p.x[3] + x;
  p.poly = p.gram + q;
  p.total = p.poly + q;
  return p;
}

cudaError_t launch_muon(const MuonArgs& a, int grad_bf16, MapEncoder enc, int num_sms, cudaStream_t s) {
  cudaError_t e = grad_bf16 ? prepare<__nv_bfloat16>(a, s) : prepare<float>(a, s);
  if (e != cudaSuccess) return e;
  // 256 x 256 tiles by pairs of CTAs where they fill the machine about twice, else
  // 128 x 128 tiles
  const long long wide = static_cast<long long>(a.L) * ((a.n + 255) / 256) * ((a.m + 255) / 256);
  return wide >= num_sms ? run_steps<2>(a, enc, num_sms, s) : run_steps<1>(a, enc, num_sms, s);
}

}  // namespace eas
