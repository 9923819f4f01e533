// Root-mean-square norm of rows with the residual's addition, and its backward.
//
//   s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),  y = (s w) rstd,
//   q = e4m3(y inv), inv = 448 / amax, scale = amax / 448, amax = max |y|.
// (s w) rstd is monotonic in |s w| for a row's rstd, so amax = max |s w| * rstd
// is the largest |y| to the bit, and the row's two statistics, sum s^2 and
// max |s w|, come from one pass and one block reduction.
//
// Backward, with g = dy w and n = s rstd:
//   dx = ds + rstd (g - s rstd^2 / H sum(g s)),   dw = sum over rows of dy n.
// rstd is recomputed from s (its row is read anyway), so the gradient is that
// of the stored s and nothing but s is kept from the forward.
//
// All of it is bound by bytes: about 10 operations an element.  What it takes is
// to have enough of them on their way all the time, which a row held by threads
// that load, reduce and store in turn does not: [65536, 5120] bf16 backward took
// 737 us that way and takes 395 with the ring below (6.8 TB/s), and [262144,
// 8192] forward with residual, mask and codes 3023 us and 2780 (6.9 TB/s).
#include <cuda_fp8.h>

#include "eas_device.cuh"
#include "eas_launch.cuh"
#include "eas_ops.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

// Rows below this amax are stored as zeros with scale 1: 448 / amax would
// leave the fp32 range (2^-117 * 2^117 * 448 is still finite).
constexpr float kTinyAmax = 6.0185e-36f;   // 2^-117

struct RowScale {
  float scale, inv;
};

__device__ __forceinline__ RowScale row_scale(float amax) {
  if (!(amax >= kTinyAmax)) return {1.f, amax > 0.f ? 0.f : 1.f};
  return {__fdiv_rn(amax, 448.f), __fdiv_rn(448.f, amax)};
}

template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&y)[VEC], float inv) {
  if constexpr (VEC == 1) {
    *p = static_cast<uint8_t>(__nv_cvt_float_to_fp8(__fmul_rn(y[0], inv), __NV_SATFINITE, __NV_E4M3));
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(__fmul_rn(y[4 * i], inv), __fmul_rn(y[4 * i + 1], inv)), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(__fmul_rn(y[4 * i + 2], inv), __fmul_rn(y[4 * i + 3], inv)), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    if constexpr (VEC == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

// ---------------------------------------------------------------- the ring
//
// The rows of a CTA run ahead in a ring in shared memory, kStages rows deep,
// filled by cp.async.  Each thread copies the 16-byte vectors that it will
// itself consume, so the ring needs no barrier; the one barrier a row is the
// reduction's.
//
// A CTA holds one row at a time, or (kShort) each of its eight warps its own
// rows, blockDim.x lanes a row.  With a mask the group lists the rows that it
// has to look at; the others are fill_rows_kernel's.
//
// Rows that do not start on 16-byte boundaries (kOdd, H no multiple of a
// vector): the vectors stay on the boundaries in memory and cover the row with
// some elements to spare at its ends, which count as zero and are not stored.
// All rows of a group start equally far from a boundary, since they lie a
// multiple of the vector's length apart, so a thread's columns stay its own.

constexpr int kListRows = 512;    // rows a group lists at a time
constexpr int kActive = 1 << 15;  // flag of a listed row
constexpr int kShortWarps = 8;

// n < 16: the rest of the 16 bytes is filled with zeros.
__device__ __forceinline__ void cp_async16(void* smem, const void* gmem, int n = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem)), "l"(gmem), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The first column of this thread's vector j; `shift` elements of a row's first
// vector lie before the row.
template <int VEC>
__device__ __forceinline__ int column(int j, int shift) {
  return static_cast<int>(j * blockDim.x + threadIdx.x) * VEC - shift;
}

// Copies vector c of the row at element `off` of src to the ring.  `bytes`: the
// length of src, which a vector past an odd row's end can reach beyond.
template <typename T, bool kOdd>
__device__ __forceinline__ void copy_vector(void* slot, const T* src, long long off, int c,
                                            long long bytes) {
  if constexpr (kOdd) {
    const long long left = bytes - (off + c) * static_cast<long long>(sizeof(T));
    cp_async16(slot, src + off + c, left < 16 ? static_cast<int>(left) : 16);
  } else {
    cp_async16(slot, src + off + c);
  }
}

template <int VEC, bool kOdd>
__device__ __forceinline__ bool whole(int c, int H) {
  return !kOdd || (c >= 0 && c + VEC <= H);
}

// A vector from the ring, widened; elements outside the row are zero.
template <typename T, int VEC, bool kOdd>
__device__ __forceinline__ void widen_row(const Raw<T, VEC>& r, int c, int H, float (&f)[VEC]) {
  widen<T, VEC>(r, f);
  if constexpr (kOdd) {
    if (!whole<VEC, kOdd>(c, H)) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (c + i < 0 || c + i >= H) f[i] = 0.f;
    }
  }
}

// Vector c of a row that starts at p (the weight).
template <typename T, int VEC, bool kOdd>
__device__ __forceinline__ Raw<T, VEC> load_row(const T* p, int c, int H) {
  if constexpr (!kOdd) return load_raw<T, VEC>(p + c);
  union {
    T t[VEC];
    Raw<T, VEC> r;
  } u = {};
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    if (c + i >= 0 && c + i < H) u.t[i] = p[c + i];
  return u.r;
}

template <typename T, int VEC, bool kOdd>
__device__ __forceinline__ void store_row(T* p, int c, int H, const float (&f)[VEC]) {
  if (whole<VEC, kOdd>(c, H)) {
    store_vec<T, VEC>(p + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float e[1] = {f[i]};
      if (c + i >= 0 && c + i < H) store_vec<T, 1>(p + c + i, e);
    }
  }
}

template <int VEC, bool kOdd>
__device__ __forceinline__ void store_row_e4m3(uint8_t* p, int c, int H, const float (&f)[VEC], float inv) {
  if (whole<VEC, kOdd>(c, H)) {
    store_e4m3<VEC>(p + c, f, inv);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float e[1] = {f[i]};
      if (c + i >= 0 && c + i < H) store_e4m3<1>(p + c + i, e, inv);
    }
  }
}

// Combines (a, b) over the threads of a row that a CTA (of two warps or more) holds:
// a by sum, b by sum or maximum.  `red` alternates with the row's parity, so one barrier a row is enough.
template <bool kMaxB>
__device__ __forceinline__ void reduce_pair(float& a, float& b, float2* red, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    const float t = __shfl_xor_sync(0xffffffffu, b, o);
    b = kMaxB ? fmaxf(b, t) : b + t;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? red[lane] : make_float2(0.f, 0.f);
  a = v.x;
  b = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    const float t = __shfl_xor_sync(0xffffffffu, b, o);
    b = kMaxB ? fmaxf(b, t) : b + t;
  }
}

// The same over the lanes of a short row.
template <bool kMaxB>
__device__ __forceinline__ void reduce_lanes(float& a, float& b) {
  for (int o = blockDim.x / 2; o > 0; o /= 2) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    const float t = __shfl_xor_sync(0xffffffffu, b, o);
    b = kMaxB ? fmaxf(b, t) : b + t;
  }
}

// A warp lists rows i of [0, span) (row first + i * step): the active ones with
// kActive set, and with `all` the others too.  Returns their number.
__device__ __forceinline__ int list_rows(unsigned short* list, const uint8_t* mask, long long first,
                                         long long step, int span, bool all) {
  const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
  int n = 0;
  for (int i0 = 0; i0 < span; i0 += 32) {
    const int i = i0 + lane;
    const bool a = i < span && mask[first + i * step] != 0;
    const bool in = a || (all && i < span);
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (in) list[n + __popc(m & ((1u << lane) - 1))] = static_cast<unsigned short>(i | (a ? kActive : 0));
    n += __popc(m);
  }
  return n;
}

// ------------------------------------------------------------------ forward

// Half of what it moves is stores, and few long-lived CTAs store at their own
// pace: the machine then writes all over its output at once.  So a CTA takes
// `batch` rows (each of its warps, kShort) and ends; the hardware hands the
// batches out in order.
template <typename T, int NV, int kStages, bool kShort, bool kOdd, bool kRes, bool kMask>
__global__ void __launch_bounds__(kShort ? 256 : 512, kShort ? (NV == 2 ? 3 : 2) : 1)
rmsnorm_fwd_ring_kernel(const RmsNormFwdArgs p, const int batch) {
  constexpr int VEC = kVec16<T>;
  launch_dependents();                  // the rows left out, on what this grid leaves free
  // [kStages][1 or 2][NV][threads].  Where it started on a 16-byte but no 128-byte
  // boundary, each cp.async fetched its sectors from L2 twice.
  extern __shared__ __align__(128) uint4 ring[];
  __shared__ float2 red[2][32];
  __shared__ int listed;
  __shared__ unsigned short list[kShort ? kShortWarps : 1][kMask ? kListRows : 1];
  const int cta = blockDim.x * blockDim.y;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int group = kShort ? warp : 0;                    // who shares a list of rows
  const int abreast = kShort ? 32 / blockDim.x : 1;       // rows a group holds at a time
  const int sub = kShort ? lane / blockDim.x : 0;
  constexpr int kArrays = kRes ? 2 : 1;
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.r);
  const long long bytes = p.R * p.H * static_cast<long long>(sizeof(T));
  const bool carry = kRes && p.s_out;                     // every row is read
  // this group's rows: first, first + 8, ...
  constexpr int kStep = 8;
  const long long unit = kShort ? static_cast<long long>(blockIdx.x) : blockIdx.x / kStep;
  const long long first = unit * kStep * batch + (kShort ? warp : static_cast<int>(blockIdx.x % kStep));
  const long long left = first < p.R ? (p.R - first + kStep - 1) / kStep : 0;
  const int span = static_cast<int>(left < batch ? left : batch);
  const int shift = kOdd ? static_cast<int>(first * p.H % VEC) : 0;
  Raw<T, VEC> rw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = column<VEC>(j, shift);
    if (c < p.H) rw[j] = load_row<T, VEC, kOdd>(static_cast<const T*>(p.w), c, p.H);
  }
  const float inv_h = 1.f / static_cast<float>(p.H);
  int parity = 0;
  int n = span;
  const unsigned short* mine = list[group];
  if constexpr (kMask) {
    if (kShort || warp == 0) {
      n = list_rows(list[group], p.mask, first, kStep, span, carry);
      if (!kShort && lane == 0) listed = n;
    }
    if constexpr (kShort) {
      __syncwarp();
    } else {
      __syncthreads();
      n = listed;
    }
  }
  auto row_at = [&](int e) -> long long { return first + kStep * (kMask ? mine[e] & (kActive - 1) : e); };
  auto issue = [&](int k) {
    const int e = k * abreast + sub;
    if (e < n) {
      const long long off = row_at(e) * p.H;
      uint4* slot = ring + static_cast<size_t>(k % kStages) * kArrays * NV * cta + tid;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = column<VEC>(j, shift);
        if (c < p.H) {
          copy_vector<T, kOdd>(slot + j * cta, x, off, c, bytes);
          if constexpr (kRes) copy_vector<T, kOdd>(slot + (NV + j) * cta, res, off, c, bytes);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue(k);

  for (int k = 0; k * abreast < n; ++k) {
    issue(k + kStages - 1);
    cp_async_wait<kStages - 1>();
    const int e = k * abreast + sub;
    const bool valid = !kShort || e < n;
    const bool active = valid && (!kMask || (mine[e] & kActive));
    const long long row = valid ? row_at(e) : 0;
    const long long off = row * p.H;
    const uint4* slot = ring + static_cast<size_t>(k % kStages) * kArrays * NV * cta + tid;
    float t[NV][VEC];
    float ss = 0.f, mx = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = column<VEC>(j, shift);
      if (c < p.H && valid) {
        widen_row<T, VEC, kOdd>(Raw<T, VEC>{slot[j * cta]}, c, p.H, t[j]);
        if constexpr (kRes) {
          float f[VEC];
          widen_row<T, VEC, kOdd>(Raw<T, VEC>{slot[(NV + j) * cta]}, c, p.H, f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) t[j][i] += f[i];
          // the stored sum is rounded once; the norm goes on with the fp32 sum
          if (carry) store_row<T, VEC, kOdd>(static_cast<T*>(p.s_out) + off, c, p.H, t[j]);
        }
        float wf[VEC];
        widen<T, VEC>(rw[j], wf);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          ss = fmaf(t[j][i], t[j][i], ss);
          t[j][i] *= wf[i];
          mx = fmaxf(mx, fabsf(t[j][i]));
        }
      }
    }
    float rstd = 0.f;
    RowScale rs = {1.f, 1.f};
    if constexpr (kShort) reduce_lanes<true>(ss, mx);
    if (!valid) continue;
    if (active) {
      if constexpr (!kShort) {
        reduce_pair<true>(ss, mx, red[parity], blockDim.x >> 5);
        parity ^= 1;
      }
      rstd = rsqrtf(fmaf(ss, inv_h, p.eps));
      rs = row_scale(mx * rstd);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = column<VEC>(j, shift);
      if (c < p.H) {
        // an inactive row is zero whatever it holds
#pragma unroll
        for (int i = 0; i < VEC; ++i) t[j][i] = !kMask || active ? t[j][i] * rstd : 0.f;
        if (p.y) store_row<T, VEC, kOdd>(static_cast<T*>(p.y) + off, c, p.H, t[j]);
        if (p.q) store_row_e4m3<VEC, kOdd>(p.q + off, c, p.H, t[j], rs.inv);
      }
    }
    if (p.q && threadIdx.x == 0) p.scale[row] = rs.scale;
  }
}

// Rows too long for the ring: two walks over the row, the second from L2 (a row
// of 2^20 fp32 elements is 4 MB).  s is stored in the second walk, each thread
// its own elements, after they have been read: it may replace x or r.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
rmsnorm_fwd_long_kernel(const RmsNormFwdArgs p) {
  __shared__ float2 red[32];
  const long long row = blockIdx.x, off = row * p.H;
  const T* x = static_cast<const T*>(p.x) + off;
  const T* r = p.r ? static_cast<const T*>(p.r) + off : nullptr;
  const T* w = static_cast<const T*>(p.w);
  T* so = p.s_out ? static_cast<T*>(p.s_out) + off : nullptr;
  const bool active = !p.mask || p.mask[row] != 0;
  auto sum = [&](int c, float (&s)[VEC]) {
    widen<T, VEC>(load_raw<T, VEC>(x + c), s);
    if (r) {
      float f[VEC];
      widen<T, VEC>(load_raw<T, VEC>(r + c), f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[i] += f[i];
    }
  };
  float ss = 0.f, mx = 0.f;
  if (active) {
#pragma unroll 2
    for (int c = threadIdx.x * VEC; c < p.H; c += blockDim.x * VEC) {
      float s[VEC], wf[VEC];
      sum(c, s);
      widen<T, VEC>(load_raw<T, VEC>(w + c), wf);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        ss = fmaf(s[i], s[i], ss);
        mx = fmaxf(mx, fabsf(s[i] * wf[i]));
      }
    }
    reduce_pair<true>(ss, mx, red, blockDim.x >> 5);
  }
  const float rstd = rsqrtf(ss / static_cast<float>(p.H) + p.eps);
  const RowScale rs = active ? row_scale(mx * rstd) : RowScale{1.f, 1.f};
  for (int c = threadIdx.x * VEC; c < p.H; c += blockDim.x * VEC) {
    float s[VEC] = {};
    if (active || so) sum(c, s);
    if (so) store_vec<T, VEC>(so + c, s);
    float wf[VEC];
    if (active) widen<T, VEC>(load_raw<T, VEC>(w + c), wf);
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[i] = active ? s[i] * wf[i] * rstd : 0.f;
    if (p.y) store_vec<T, VEC>(static_cast<T*>(p.y) + off + c, s);
    if (p.q) store_e4m3<VEC>(p.q + off + c, s, rs.inv);
  }
  if (p.q && threadIdx.x == 0) p.scale[row] = rs.scale;
}

// ----------------------------------------------------------------- backward

// Each thread keeps its columns' share of dw in registers and adds it to the
// CTA's row of `partial` at the end.  The number of partial rows and the order
// of every sum depend on the shape and the machine only, so results repeat to
// the bit.  Whether there is a ds and a mask is compiled in for the longer
// rows: [65536, 5120] bf16 with ds took 447 us deciding in the loop and 395
// without.
template <typename T, int NV, int kStages, bool kShort, bool kOdd, bool kDs, bool kMask>
__global__ void __launch_bounds__(kShort ? 256 : 512, kShort ? 2 : 1)
rmsnorm_bwd_ring_kernel(const RmsNormBwdArgs p) {
  constexpr int VEC = kVec16<T>;
  launch_dependents();
  extern __shared__ __align__(128) uint4 ring[];  // [kStages][2 or 3][NV][threads]
  __shared__ float2 red[2][32];
  __shared__ int listed;
  __shared__ unsigned short list[kShort ? kShortWarps : 1][kMask || kShort ? kListRows : 1];
  const int cta = blockDim.x * blockDim.y;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int group = kShort ? warp : 0;
  const int groups = kShort ? kShortWarps : 1;
  const int abreast = kShort ? 32 / blockDim.x : 1;
  const int sub = kShort ? lane / blockDim.x : 0;
  // short rows decide while they run
  const bool with_ds = kShort ? p.ds != nullptr : kDs;
  const bool masked = kShort ? p.mask != nullptr : kMask;
  const int arrays = with_ds ? 3 : 2;
  const T* dy = static_cast<const T*>(p.dy);
  const T* sv = static_cast<const T*>(p.s);
  const T* ds = static_cast<const T*>(p.ds);
  T* dx = static_cast<T*>(p.dx);
  const long long bytes = p.R * p.H * static_cast<long long>(sizeof(T));
  const long long first = static_cast<long long>(blockIdx.x) * groups + group;
  const long long step = static_cast<long long>(gridDim.x) * groups;
  const long long rows = first < p.R ? (p.R - first + step - 1) / step : 0;
  const int shift = kOdd ? static_cast<int>(first * p.H % VEC) : 0;
  Raw<T, VEC> rw[NV];
  float acc[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = column<VEC>(j, shift);
    if (c < p.H) rw[j] = load_row<T, VEC, kOdd>(static_cast<const T*>(p.w), c, p.H);
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
  }
  const float inv_h = 1.f / static_cast<float>(p.H);
  int parity = 0;

  for (long long base = 0; base < rows; base += kListRows) {
    const int span = static_cast<int>(rows - base < kListRows ? rows - base : kListRows);
    int n = span;
    const unsigned short* mine = list[group];
    if (masked) {
      if (kShort || warp == 0) {
        n = list_rows(list[group], p.mask, first + base * step, step, span, false);
        if (!kShort && lane == 0) listed = n;
      }
      if constexpr (kShort) {
        __syncwarp();
      } else {
        __syncthreads();
        n = listed;
      }
    }
    auto row_at = [&](int e) -> long long {
      return first + (base + (masked ? mine[e] & (kActive - 1) : e)) * step;
    };
    auto issue = [&](int k) {
      const int e = k * abreast + sub;
      if (e < n) {
        const long long off = row_at(e) * p.H;
        uint4* slot = ring + static_cast<size_t>(k % kStages) * arrays * NV * cta + tid;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = column<VEC>(j, shift);
          if (c < p.H) {
            copy_vector<T, kOdd>(slot + j * cta, dy, off, c, bytes);
            copy_vector<T, kOdd>(slot + (NV + j) * cta, sv, off, c, bytes);
            if (with_ds) copy_vector<T, kOdd>(slot + (2 * NV + j) * cta, ds, off, c, bytes);
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k);

    for (int k = 0; k * abreast < n; ++k) {
      issue(k + kStages - 1);
      cp_async_wait<kStages - 1>();
      const int e = k * abreast + sub;
      const bool valid = !kShort || e < n;
      const long long off = valid ? row_at(e) * p.H : 0;
      const uint4* slot = ring + static_cast<size_t>(k % kStages) * arrays * NV * cta + tid;
      Raw<T, VEC> rdy[NV], rsv[NV];
      float ss = 0.f, gs = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = column<VEC>(j, shift);
        if (c < p.H && valid) {
          rdy[j].v = slot[j * cta];
          rsv[j].v = slot[(NV + j) * cta];
          float s[VEC], d[VEC], wf[VEC];
          widen_row<T, VEC, kOdd>(rsv[j], c, p.H, s);
          widen_row<T, VEC, kOdd>(rdy[j], c, p.H, d);
          widen<T, VEC>(rw[j], wf);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            ss = fmaf(s[i], s[i], ss);
            gs = fmaf(d[i] * wf[i], s[i], gs);
          }
        }
      }
      if constexpr (kShort) {
        reduce_lanes<false>(ss, gs);
      } else {
        reduce_pair<false>(ss, gs, red[parity], blockDim.x >> 5);
        parity ^= 1;
      }
      if (!valid) continue;
      const float rstd = rsqrtf(fmaf(ss, inv_h, p.eps));
      const float c2 = gs * rstd * rstd * inv_h;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = column<VEC>(j, shift);
        if (c < p.H) {
          float s[VEC], d[VEC], wf[VEC], o[VEC] = {};
          widen_row<T, VEC, kOdd>(rsv[j], c, p.H, s);
          widen_row<T, VEC, kOdd>(rdy[j], c, p.H, d);
          widen<T, VEC>(rw[j], wf);
          if (with_ds) widen<T, VEC>(Raw<T, VEC>{slot[(2 * NV + j) * cta]}, o);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            o[i] = fmaf(rstd, fmaf(-s[i], c2, d[i] * wf[i]), o[i]);
            acc[j][i] = fmaf(d[i], s[i] * rstd, acc[j][i]);
          }
          store_row<T, VEC, kOdd>(dx + off, c, p.H, o);
        }
      }
    }
    cp_async_wait<0>();
    if (base + kListRows < rows) {
      if constexpr (kShort) __syncwarp(); else __syncthreads();
    }
  }

  float* out = p.partial + static_cast<long long>(blockIdx.x) * p.H;
  if constexpr (kShort) {
    // lanes that hold the same columns, then the warps in order (the ring, whose
    // copies have all landed, is at least as large as the warps' sums)
    __syncthreads();
    float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = column<VEC>(j, shift);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        for (int o = blockDim.x; o < 32; o *= 2) acc[j][i] += __shfl_xor_sync(0xffffffffu, acc[j][i], o);
        if (sub == 0 && c + i >= 0 && c + i < p.H) sums[warp * p.H + c + i] = acc[j][i];
      }
    }
    __syncthreads();
    for (int c = tid; c < p.H; c += cta) {
      float t = sums[c];
#pragma unroll
      for (int g = 1; g < kShortWarps; ++g) t += sums[g * p.H + c];
      out[c] = t;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = column<VEC>(j, shift);
      if (c >= p.H) continue;
#pragma unroll
      for (int h = 0; h < VEC; h += 4) {
        if constexpr (kOdd) {
#pragma unroll
          for (int i = h; i < h + 4; ++i)
            if (c + i >= 0 && c + i < p.H) out[c + i] = acc[j][i];
        } else {
          *reinterpret_cast<float4*>(out + c + h) =
              make_float4(acc[j][h], acc[j][h + 1], acc[j][h + 2], acc[j][h + 3]);
        }
      }
    }
  }
}

// The inactive rows that a ring kernel leaves out; it runs beside that one.
// dst = src or zero on them, and in the forward also q = 0 and scale = 1.  Small
// CTAs in the order of the rows: where the ring kernel's CTAs wrote these rows
// themselves, one a SM and each at its own pace, the backward of [131072, 7168]
// bf16 with 10 % active rows took 388 us against 340.
struct FillArgs {
  const char* src;        // or null: zeros
  char* dst;              // or null
  uint8_t* q;             // or null
  float* scale;           // with q
  const uint8_t* mask;
  long long R;
  int row_bytes;          // of src and dst
  int H;                  // row bytes of q
  int rows;               // rows of a CTA
};

// n bytes of dst from src (which lies as dst does to 16 bytes) or zero.
__device__ __forceinline__ void fill_bytes(char* dst, const char* src, int n) {
  int head = static_cast<int>(-reinterpret_cast<uintptr_t>(dst) & 15);
  if (head > n) head = n;
  const int mid = (n - head) & ~15;
#pragma unroll 4
  for (int b = threadIdx.x * 16; b < mid; b += blockDim.x * 16)
    *reinterpret_cast<uint4*>(dst + head + b) =
        src ? *reinterpret_cast<const uint4*>(src + head + b) : make_uint4(0, 0, 0, 0);
  for (int b = threadIdx.x; b < n - mid; b += blockDim.x) {
    const int at = b < head ? b : mid + b;
    dst[at] = src ? src[at] : 0;
  }
}

__global__ void __launch_bounds__(256) fill_rows_kernel(const FillArgs p) {
  const long long r0 = static_cast<long long>(blockIdx.x) * p.rows;
  for (int r = threadIdx.y; r < p.rows && r0 + r < p.R; r += blockDim.y) {
    const long long row = r0 + r;
    if (p.mask[row] != 0) continue;
    const long long off = row * p.row_bytes;
    if (p.dst) fill_bytes(p.dst + off, p.src ? p.src + off : nullptr, p.row_bytes);
    if (p.q) {
      fill_bytes(reinterpret_cast<char*>(p.q) + row * p.H, nullptr, p.H);
      if (threadIdx.x == 0) p.scale[row] = 1.f;
    }
  }
  wait_for_launch_before();   // whoever waits for this launch waits for the ring kernel too
}

cudaError_t launch_fill(FillArgs f, cudaStream_t s) {
  f.rows = 65536 / f.row_bytes < 1 ? 1 : 65536 / f.row_bytes < 256 ? 65536 / f.row_bytes : 256;
  int tx = 16;
  while (tx < 256 && tx * 16 < f.row_bytes) tx *= 2;
  const long long grid = (f.R + f.rows - 1) / f.rows;
  return launch_overlapped(fill_rows_kernel, dim3(static_cast<unsigned>(grid)), dim3(tx, 256 / tx), 0,
                           s, f);
}

// Rows too long for the ring: dx in two walks of the row, the row's rstd kept
// for the dw pass.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
rmsnorm_bwd_long_kernel(const RmsNormBwdArgs p) {
  __shared__ float2 red[32];
  const long long row = blockIdx.x, off = row * p.H;
  const T* dy = static_cast<const T*>(p.dy) + off;
  const T* sp = static_cast<const T*>(p.s) + off;
  const T* w = static_cast<const T*>(p.w);
  const T* ds = p.ds ? static_cast<const T*>(p.ds) + off : nullptr;
  T* dx = static_cast<T*>(p.dx) + off;
  const bool active = !p.mask || p.mask[row] != 0;
  float ss = 0.f, gs = 0.f;
  if (active) {
#pragma unroll 2
    for (int c = threadIdx.x * VEC; c < p.H; c += blockDim.x * VEC) {
      float s[VEC], d[VEC], wf[VEC];
      widen<T, VEC>(load_raw<T, VEC>(sp + c), s);
      widen<T, VEC>(load_raw<T, VEC>(dy + c), d);
      widen<T, VEC>(load_raw<T, VEC>(w + c), wf);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        ss = fmaf(s[i], s[i], ss);
        gs = fmaf(d[i] * wf[i], s[i], gs);
      }
    }
    reduce_pair<false>(ss, gs, red, blockDim.x >> 5);
  }
  const float inv_h = 1.f / static_cast<float>(p.H);
  const float rstd = rsqrtf(fmaf(ss, inv_h, p.eps));
  const float c2 = gs * rstd * rstd * inv_h;
  for (int c = threadIdx.x * VEC; c < p.H; c += blockDim.x * VEC) {
    float o[VEC] = {};
    if (ds) widen<T, VEC>(load_raw<T, VEC>(ds + c), o);
    if (active) {
      float s[VEC], d[VEC], wf[VEC];
      widen<T, VEC>(load_raw<T, VEC>(sp + c), s);
      widen<T, VEC>(load_raw<T, VEC>(dy + c), d);
      widen<T, VEC>(load_raw<T, VEC>(w + c), wf);
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = fmaf(rstd, fmaf(-s[i], c2, d[i] * wf[i]), o[i]);
    }
    store_vec<T, VEC>(dx + c, o);
  }
  if (threadIdx.x == 0) p.rstd[row] = active ? rstd : 0.f;
}

// dw partials of long rows: CTA (x, y) sums columns [256 x, 256 x + 256) over
// the rows y, y + gridDim.y, ...; inactive rows are not read.
template <typename T>
__global__ void __launch_bounds__(256)
rmsnorm_dw_long_kernel(const RmsNormBwdArgs p) {
  const long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= p.H) return;
  float acc = 0.f;
  for (long long row = blockIdx.y; row < p.R; row += gridDim.y)
    if (!p.mask || p.mask[row] != 0)
      acc = fmaf(to_f32(static_cast<const T*>(p.dy)[row * p.H + c]),
                 to_f32(static_cast<const T*>(p.s)[row * p.H + c]) * p.rstd[row], acc);
  p.partial[static_cast<long long>(blockIdx.y) * p.H + c] = acc;
}

// dw[c] = sum of the partial rows in a fixed order: 32 columns a CTA, its
// warps take every kDwWarps-th partial row, then the warps' sums in order.
constexpr int kDwWarps = 16;
__global__ void __launch_bounds__(32 * kDwWarps)
rmsnorm_dw_kernel(const float* partial, int n, int H, float* dw, DevStatus* st) {
  __shared__ float sm[kDwWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.f;
  wait_for_launch_before();
  if (blockIdx.x == 0 && threadIdx.x == 0) *st = DevStatus{};   // nothing here can fail on the device
  if (c < H) {
#pragma unroll 8
    for (int i = warp; i < n; i += kDwWarps) acc += partial[static_cast<long long>(i) * H + c];
  }
  sm[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < kDwWarps; ++i) acc += sm[i][lane];
    dw[c] = acc;
  }
}

// --------------------------------------------------------------- row shapes

// How a ring kernel holds rows of H elements; stages 0: too long for it.
struct RingShape {
  bool odd;                // rows do not start on 16-byte boundaries
  int nv;                  // vectors a thread
  int lanes, groups;       // block (lanes, groups); groups > 1: rows within warps
  int ctas, stages;
  size_t smem;
};

// About 512 threads an SM, two or four vectors each: the backward of [65536,
// 8192] bf16 with ds took 742 us with one row by 1024 threads of one vector and
// 600 by 512 of two.  Three rows deep: 600 us against 630 with two and 639 with
// four; at [65536, 4096] fp32 477 against 508 and 525.  Rows of up to 96 vectors
// lie within warps, in lanes that they fill best: the backward of [131072, 320]
// bf16 with ds 59 us on 16 lanes of three vectors against 76 on 32 of two; above
// that a CTA of 64 lanes does better ([131072, 1024]: 170 against 180).
RingShape ring_shape(int H, int esize, int arrays) {
  RingShape r = {};
  const int vec = 16 / esize;
  r.odd = H % vec != 0;
  const int n = r.odd ? (H + 2 * vec - 2) / vec : H / vec;   // vectors that cover a row anywhere
  if (n > 2048) return r;
  r.groups = 1;
  if (n <= 96) {                        // rows within warps: the lanes that n fills best
    r.lanes = n <= 24 ? 8 : n <= 48 ? 16 : 32;
    r.nv = n <= 2 * r.lanes ? 2 : 3;
    r.groups = 32 * kShortWarps / r.lanes;
  } else {
    r.nv = n <= 1024 ? 2 : 4;
    r.lanes = ((n + r.nv - 1) / r.nv + 31) / 32 * 32;
  }
  const int cta = r.lanes * r.groups;
  r.ctas = cta < 512 ? 512 / cta : 1;
  const size_t stage = static_cast<size_t>(arrays) * r.nv * cta * 16;
  r.stages = r.ctas * 3 * stage <= 200u << 10 ? 3 : 2;
  r.smem = r.stages * stage;
  return r;
}

// The most shared memory that ring_shape asks for: three stages fit 200 KB on all
// of an SM's CTAs, and two of the largest (three arrays of 2048 vectors) take 192.
constexpr int kRingBytes = 200 << 10;

template <auto kKernel, typename... A>
cudaError_t ring_launch(const RingShape& r, unsigned grid, cudaStream_t s, A... args) {
  if (r.smem > kRingBytes) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<kKernel>(kRingBytes);
  if (e != cudaSuccess) return e;
  kKernel<<<grid, dim3(r.lanes, r.groups), r.smem, s>>>(args...);
  return cudaGetLastError();
}

template <typename T, int NV, bool kShort, bool kOdd>
cudaError_t fwd_kind(const RmsNormFwdArgs& a, const RingShape& r, cudaStream_t s, int batch,
                     unsigned g) {
  if (a.r)
    return a.mask ? ring_launch<rmsnorm_fwd_ring_kernel<T, NV, 3, kShort, kOdd, true, true>>(r, g, s, a, batch)
                  : ring_launch<rmsnorm_fwd_ring_kernel<T, NV, 3, kShort, kOdd, true, false>>(r, g, s, a, batch);
  return a.mask ? ring_launch<rmsnorm_fwd_ring_kernel<T, NV, 3, kShort, kOdd, false, true>>(r, g, s, a, batch)
                : ring_launch<rmsnorm_fwd_ring_kernel<T, NV, 3, kShort, kOdd, false, false>>(r, g, s, a, batch);
}

template <typename T, bool kOdd>
cudaError_t fwd_rows(const RmsNormFwdArgs& a, const RingShape& r, cudaStream_t s, int batch,
                     unsigned g) {
  if (r.groups > 1)
    return r.nv == 2 ? fwd_kind<T, 2, true, kOdd>(a, r, s, batch, g) : fwd_kind<T, 3, true, kOdd>(a, r, s, batch, g);
  return r.nv == 2 ? fwd_kind<T, 2, false, kOdd>(a, r, s, batch, g) : fwd_kind<T, 4, false, kOdd>(a, r, s, batch, g);
}

template <typename T>
cudaError_t fwd_t(const RmsNormFwdArgs& a, int num_sms, cudaStream_t s) {
  RingShape r = ring_shape(a.H, sizeof(T), a.r ? 2 : 1);
  if (r.stages == 0) {
    const unsigned grid = static_cast<unsigned>(a.R);
    if (r.odd) rmsnorm_fwd_long_kernel<T, 1><<<grid, 1024, 0, s>>>(a);
    else rmsnorm_fwd_long_kernel<T, kVec16<T>><<<grid, 1024, 0, s>>>(a);
    return cudaGetLastError();
  }
  r.smem = r.smem / r.stages * 3;       // always three rows deep: at most 192 KB
  // As many rows as leave 32 batches an SM, eight at most ([262144, 8192] bf16
  // with residual and codes: one row 4600 us, two 3390, four 2910, eight 2776;
  // without end, two CTAs an SM, 3027).  Narrow rows go abreast, so eight each.
  int batch = 1;
  const int most = 8 * (r.groups > 1 ? 32 / r.lanes : 1);
  while (batch < most && a.R >= 32LL * num_sms * batch * (r.groups > 1 ? kShortWarps : 1)) batch *= 2;
  const long long units = (a.R + 8LL * batch - 1) / (8LL * batch);   // of 8 batches
  const unsigned g = static_cast<unsigned>(r.groups > 1 ? units : batch == 1 ? a.R : 8 * units);
  const cudaError_t e = r.odd ? fwd_rows<T, true>(a, r, s, batch, g) : fwd_rows<T, false>(a, r, s, batch, g);
  if (e != cudaSuccess || !a.mask || (a.r && a.s_out)) return e;   // every row was read
  return launch_fill({nullptr, static_cast<char*>(a.y), a.q, a.scale, a.mask, a.R,
                      a.H * static_cast<int>(sizeof(T)), a.H, 0}, s);
}

template <typename T, int NV, int S, bool kOdd>
cudaError_t bwd_kind(const RmsNormBwdArgs& a, const RingShape& r, unsigned g, cudaStream_t s) {
  if (a.ds)
    return a.mask ? ring_launch<rmsnorm_bwd_ring_kernel<T, NV, S, false, kOdd, true, true>>(r, g, s, a)
                  : ring_launch<rmsnorm_bwd_ring_kernel<T, NV, S, false, kOdd, true, false>>(r, g, s, a);
  return a.mask ? ring_launch<rmsnorm_bwd_ring_kernel<T, NV, S, false, kOdd, false, true>>(r, g, s, a)
                : ring_launch<rmsnorm_bwd_ring_kernel<T, NV, S, false, kOdd, false, false>>(r, g, s, a);
}

template <typename T, int NV, int S, bool kOdd>
cudaError_t bwd_short(const RmsNormBwdArgs& a, const RingShape& r, unsigned g, cudaStream_t s) {
  return ring_launch<rmsnorm_bwd_ring_kernel<T, NV, S, true, kOdd, false, false>>(r, g, s, a);
}

template <typename T, bool kOdd>
cudaError_t bwd_rows(const RmsNormBwdArgs& a, const RingShape& r, unsigned g, cudaStream_t s) {
  if (r.groups > 1) {
    if (r.nv == 2) return bwd_short<T, 2, 3, kOdd>(a, r, g, s);
    return r.stages == 2 ? bwd_short<T, 3, 2, kOdd>(a, r, g, s) : bwd_short<T, 3, 3, kOdd>(a, r, g, s);
  }
  if (r.nv == 2) return bwd_kind<T, 2, 3, kOdd>(a, r, g, s);   // 512 threads an SM: always three deep
  return r.stages == 2 ? bwd_kind<T, 4, 2, kOdd>(a, r, g, s) : bwd_kind<T, 4, 3, kOdd>(a, r, g, s);
}

template <typename T>
cudaError_t bwd_t(const RmsNormBwdArgs& a, int num_sms, int* n_partials, cudaStream_t s) {
  const long long most = rmsnorm_bwd_partials(a.R, a.H);
  const RingShape r = ring_shape(a.H, sizeof(T), a.ds ? 3 : 2);
  if (r.stages == 0) {
    const int splits = static_cast<int>(most < 32 ? most : 32);
    if (a.R > 0) {
      const unsigned grid = static_cast<unsigned>(a.R);
      if (r.odd) rmsnorm_bwd_long_kernel<T, 1><<<grid, 1024, 0, s>>>(a);
      else rmsnorm_bwd_long_kernel<T, kVec16<T>><<<grid, 1024, 0, s>>>(a);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    rmsnorm_dw_long_kernel<T><<<dim3((a.H + 255) / 256, splits), 256, 0, s>>>(a);
    *n_partials = splits;
    return cudaGetLastError();
  }
  const int abreast = r.groups > 1 ? kShortWarps : 1;
  const long long need = (a.R + abreast - 1) / abreast;       // CTAs that have a row
  long long grid = static_cast<long long>(num_sms) * r.ctas;
  if (grid > most) grid = most;
  if (grid >= need) grid = need > 0 ? need : 1;
  else if (grid >= 8) grid -= grid % 8;                       // odd rows: a group's lie 8 k apart
  *n_partials = static_cast<int>(grid);
  const unsigned g = static_cast<unsigned>(grid);
  const cudaError_t e = r.odd ? bwd_rows<T, true>(a, r, g, s) : bwd_rows<T, false>(a, r, g, s);
  if (e != cudaSuccess || !a.mask || a.ds == a.dx || a.R == 0) return e;   // in place: ds is there
  return launch_fill({static_cast<const char*>(a.ds), static_cast<char*>(a.dx), nullptr, nullptr, a.mask,
                      a.R, a.H * static_cast<int>(sizeof(T)), a.H, 0}, s);
}

}  // namespace

// Partial rows of dw that the backward writes at most, for any machine size.
long long rmsnorm_bwd_partials(long long R, long long H) {
  const long long most = H <= 16384 ? 1024 : 32;
  return R < 1 ? 1 : R < most ? R : most;
}

cudaError_t launch_rmsnorm_fwd(const RmsNormFwdArgs& a, int is_bf16, int num_sms, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  return is_bf16 ? fwd_t<__nv_bfloat16>(a, num_sms, s) : fwd_t<float>(a, num_sms, s);
}

cudaError_t launch_rmsnorm_bwd(const RmsNormBwdArgs& a, int is_bf16, int num_sms, int* n_partials,
                               cudaStream_t s) {
  return is_bf16 ? bwd_t<__nv_bfloat16>(a, num_sms, n_partials, s)
                 : bwd_t<float>(a, num_sms, n_partials, s);
}

cudaError_t launch_rmsnorm_dw(const float* partial, int n, int H, float* dw, DevStatus* st,
                              cudaStream_t s) {
  return launch_overlapped(rmsnorm_dw_kernel, dim3((H + 31) / 32), dim3(32 * kDwWarps), 0, s, partial,
                           n, H, dw, st);
}

}  // namespace eas
