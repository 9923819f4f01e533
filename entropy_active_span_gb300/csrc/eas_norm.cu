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
// All of it is bound by bytes: about 10 operations an element.
#include <cuda_fp8.h>

#include "eas_device.cuh"
#include "eas_kernels.h"
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

// Combines (a, b) over the G threads of a row: a by sum, b by sum or maximum.
// A group is a warp (G = 32, no barrier) or the whole CTA; `red` alternates
// with the row's parity, so one barrier a row is enough.
template <bool kMaxB>
__device__ __forceinline__ void reduce_pair(float& a, float& b, float2* red, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    const float t = __shfl_xor_sync(0xffffffffu, b, o);
    b = kMaxB ? fmaxf(b, t) : b + t;
  }
  if (warps == 1) return;
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

// ------------------------------------------------------------------ forward

// One row by blockDim.x threads, blockDim.y rows a CTA (blockDim.y > 1 only
// where a warp holds a row).  The row stays in registers: NV vectors of VEC
// elements a thread, thread-contiguous so that every access is coalesced.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024)
rmsnorm_fwd_kernel(const RmsNormFwdArgs p) {
  __shared__ float2 red[32];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= p.R) return;   // whole warps: a group of several warps is the CTA
  const T* x = static_cast<const T*>(p.x) + row * p.H;
  const T* r = p.r ? static_cast<const T*>(p.r) + row * p.H : nullptr;
  const T* w = static_cast<const T*>(p.w);
  const bool active = !p.mask || p.mask[row] != 0;

  float s[NV][VEC];
  if (active || (r && p.s_out)) {
    Raw<T, VEC> rx[NV], rr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (c < p.H) {
        rx[j] = load_raw<T, VEC>(x + c);
        if (r) rr[j] = load_raw<T, VEC>(r + c);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (c < p.H) {
        widen<T, VEC>(rx[j], s[j]);
        if (r) {
          float t[VEC];
          widen<T, VEC>(rr[j], t);
#pragma unroll
          for (int i = 0; i < VEC; ++i) s[j][i] += t[i];
          // the stored sum is rounded once; the norm goes on with the fp32 sum
          if (p.s_out) store_vec<T, VEC>(static_cast<T*>(p.s_out) + row * p.H + c, s[j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[j][i] = 0.f;
      }
    }
  }
  if (!active) {
    const float z[VEC] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (c < p.H) {
        if (p.y) store_vec<T, VEC>(static_cast<T*>(p.y) + row * p.H + c, z);
        if (p.q) store_e4m3<VEC>(p.q + row * p.H + c, z, 1.f);
      }
    }
    if (p.q && threadIdx.x == 0) p.scale[row] = 1.f;
    return;
  }
  float ss = 0.f, mx = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * VEC;
    if (c < p.H) {
      float wf[VEC];
      widen<T, VEC>(load_raw<T, VEC>(w + c), wf);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        ss = fmaf(s[j][i], s[j][i], ss);
        s[j][i] *= wf[i];
        mx = fmaxf(mx, fabsf(s[j][i]));
      }
    }
  }
  reduce_pair<true>(ss, mx, red, blockDim.x >> 5);
  const float rstd = rsqrtf(ss / static_cast<float>(p.H) + p.eps);
  const RowScale rs = row_scale(mx * rstd);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * VEC;
    if (c < p.H) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[j][i] *= rstd;
      if (p.y) store_vec<T, VEC>(static_cast<T*>(p.y) + row * p.H + c, s[j]);
      if (p.q) store_e4m3<VEC>(p.q + row * p.H + c, s[j], rs.inv);
    }
  }
  if (p.q && threadIdx.x == 0) p.scale[row] = rs.scale;
}

// Rows too long for the registers of a CTA: two walks over the row, the second
// from L2 (a row of 2^20 fp32 elements is 4 MB).  One CTA of 1024 threads a
// row, element by element.  x and r are read again in the second walk, after s
// may have replaced one of them, so with r it reads what it needs first and
// stores s last, each thread its own elements.
template <typename T>
__global__ void __launch_bounds__(1024)
rmsnorm_fwd_long_kernel(const RmsNormFwdArgs p) {
  __shared__ float2 red[32];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.H;
  const T* r = p.r ? static_cast<const T*>(p.r) + row * p.H : nullptr;
  const T* w = static_cast<const T*>(p.w);
  T* so = p.s_out ? static_cast<T*>(p.s_out) + row * p.H : nullptr;
  const bool active = !p.mask || p.mask[row] != 0;
  float ss = 0.f, mx = 0.f;
  if (active) {
    for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
      const float s = to_f32(x[c]) + (r ? to_f32(r[c]) : 0.f);
      ss = fmaf(s, s, ss);
      mx = fmaxf(mx, fabsf(s * to_f32(w[c])));
    }
    reduce_pair<true>(ss, mx, red, blockDim.x >> 5);
  }
  const float rstd = rsqrtf(ss / static_cast<float>(p.H) + p.eps);
  const RowScale rs = active ? row_scale(mx * rstd) : RowScale{1.f, 1.f};
  for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
    float y[1] = {0.f};
    if (active || (r && so)) {
      const float s[1] = {to_f32(x[c]) + (r ? to_f32(r[c]) : 0.f)};
      if (active) y[0] = s[0] * to_f32(w[c]) * rstd;
      if (r && so) store_vec<T, 1>(so + c, s);
    }
    if (p.y) store_vec<T, 1>(static_cast<T*>(p.y) + row * p.H + c, y);
    if (p.q) store_e4m3<1>(p.q + row * p.H + c, y, rs.inv);
  }
  if (p.q && threadIdx.x == 0) p.scale[row] = rs.scale;
}

// ----------------------------------------------------------------- backward

// Rows that the ring kernel below does not take (unaligned ones, and beyond 32 KB).
// A CTA walks rows blockIdx.x, blockIdx.x + gridDim.x, ... (blockDim.y rows at a
// time where a warp holds a row); each thread keeps its columns' share of dw
// in registers and adds it to the CTA's row of `partial` at the end.  The
// number of partial rows and the order of every sum depend on the shape and
// the machine only, so results repeat to the bit.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024)
rmsnorm_bwd_kernel(const RmsNormBwdArgs p) {
  __shared__ float2 red[2][32];
  const T* w = static_cast<const T*>(p.w);
  Raw<T, VEC> rw[NV];
  float acc[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * VEC;
    if (c < p.H) rw[j] = load_raw<T, VEC>(w + c);
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
  }
  const float inv_h = 1.f / static_cast<float>(p.H);
  int parity = 0;
  const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
  for (long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y; row < p.R;
       row += step) {
    const T* ds = p.ds ? static_cast<const T*>(p.ds) + row * p.H : nullptr;
    T* dx = static_cast<T*>(p.dx) + row * p.H;
    if (p.mask && p.mask[row] == 0) {   // the same for every thread of the group
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
        if (c < p.H) {
          float d[VEC] = {};
          if (ds) widen<T, VEC>(load_raw<T, VEC>(ds + c), d);
          store_vec<T, VEC>(dx + c, d);
        }
      }
      continue;
    }
    const T* dy = static_cast<const T*>(p.dy) + row * p.H;
    const T* sp = static_cast<const T*>(p.s) + row * p.H;
    Raw<T, VEC> rdy[NV], rsv[NV], rds[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (c < p.H) {
        rdy[j] = load_raw<T, VEC>(dy + c);
        rsv[j] = load_raw<T, VEC>(sp + c);
        if (ds) rds[j] = load_raw<T, VEC>(ds + c);
      }
    }
    float ss = 0.f, gs = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (c < p.H) {
        float s[VEC], d[VEC], wf[VEC];
        widen<T, VEC>(rsv[j], s);
        widen<T, VEC>(rdy[j], d);
        widen<T, VEC>(rw[j], wf);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          ss = fmaf(s[i], s[i], ss);
          gs = fmaf(d[i] * wf[i], s[i], gs);
        }
      }
    }
    reduce_pair<false>(ss, gs, red[parity], blockDim.x >> 5);
    parity ^= 1;
    const float rstd = rsqrtf(fmaf(ss, inv_h, p.eps));
    const float c2 = gs * rstd * rstd * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (c < p.H) {
        float s[VEC], d[VEC], wf[VEC], o[VEC] = {};
        widen<T, VEC>(rsv[j], s);
        widen<T, VEC>(rdy[j], d);
        widen<T, VEC>(rw[j], wf);
        if (ds) widen<T, VEC>(rds[j], o);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          o[i] = fmaf(rstd, fmaf(-s[i], c2, d[i] * wf[i]), o[i]);
          acc[j][i] = fmaf(d[i], s[i] * rstd, acc[j][i]);
        }
        store_vec<T, VEC>(dx + c, o);
      }
    }
  }
  // one partial row a group: blockIdx.x * blockDim.y + threadIdx.y
  float* out = p.partial + (static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y) * p.H;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * VEC;
    if (c < p.H) store_vec<float, VEC == 1 ? 1 : 4>(out + c, *reinterpret_cast<float(*)[VEC == 1 ? 1 : 4]>(&acc[j][0]));
    if constexpr (VEC == 8)
      if (c < p.H) store_vec<float, 4>(out + c + 4, *reinterpret_cast<float(*)[4]>(&acc[j][4]));
  }
}

// The same for aligned rows, with the loads running ahead: each thread copies
// the vectors that it will itself consume into its own slots of a ring in
// shared memory, kStages rows deep, with cp.async.  A thread waits for its own
// copies only, so the ring needs no barrier; the one barrier a row is the
// reduction's.  With a mask the group lists its active rows, and the ring holds
// those alone; the others are norm_bwd_fill_kernel's.
//
// A CTA holds one row at a time, or (kShort) each of its eight warps its own
// rows, blockDim.x lanes a row.  Whether there is a ds and a mask is compiled in
// for the longer rows: [65536, 5120] bf16 with ds took 447 us deciding in the
// loop and 397 without.
__device__ __forceinline__ void cp_async16(void* smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kListRows = 512;    // rows a group lists at a time
constexpr int kShortWarps = 8;

template <typename T, int NV, int kStages, bool kShort, bool kDs, bool kMask>
__global__ void __launch_bounds__(kShort ? 256 : 512, kShort ? 2 : 1)
rmsnorm_bwd_ring_kernel(const RmsNormBwdArgs p) {
  constexpr int VEC = kVec16<T>;
  launch_dependents();                  // the rows left out, on what this grid leaves free
  // [kStages][2 or 3][NV][threads of the CTA].  Where it started on a 16-byte
  // but no 128-byte boundary, each cp.async fetched its sectors from L2 twice.
  extern __shared__ __align__(128) uint4 ring[];
  __shared__ float2 red[2][32];
  __shared__ int listed;
  __shared__ unsigned short list[kShort ? kShortWarps : 1][kListRows];
  const int cta = blockDim.x * blockDim.y;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int group = kShort ? warp : 0;                    // who shares a list of rows
  const int groups = kShort ? kShortWarps : 1;
  const int abreast = kShort ? 32 / blockDim.x : 1;       // rows a group holds at a time
  const int sub = kShort ? lane / blockDim.x : 0;
  // short rows decide while they run
  const bool with_ds = kShort ? p.ds != nullptr : kDs;
  const bool masked = kShort ? p.mask != nullptr : kMask;
  const int arrays = with_ds ? 3 : 2;
  const T* dy = static_cast<const T*>(p.dy);
  const T* sv = static_cast<const T*>(p.s);
  const T* ds = static_cast<const T*>(p.ds);
  T* dx = static_cast<T*>(p.dx);
  const T* w = static_cast<const T*>(p.w);
  Raw<T, VEC> rw[NV];
  float acc[NV][VEC];
  bool in[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * blockDim.x + threadIdx.x) * VEC;
    in[j] = c < p.H;
    if (in[j]) rw[j] = load_raw<T, VEC>(w + c);
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
  }
  const float inv_h = 1.f / static_cast<float>(p.H);
  // this group's rows: first, first + step, ...
  const long long first = static_cast<long long>(blockIdx.x) * groups + group;
  const long long step = static_cast<long long>(gridDim.x) * groups;
  const long long rows = first < p.R ? (p.R - first + step - 1) / step : 0;
  int parity = 0;

  for (long long base = 0; base < rows; base += kListRows) {
    const int span = static_cast<int>(rows - base < kListRows ? rows - base : kListRows);
    int n = span;
    unsigned short* mine = list[group];
    if (masked) {
      // a warp of the group lists the active rows
      if (kShort || warp == 0) {
        int on = 0;
        for (int i0 = 0; i0 < span; i0 += 32) {
          const int i = i0 + lane;
          const bool a = i < span && p.mask[first + (base + i) * step] != 0;
          const unsigned m = __ballot_sync(0xffffffffu, a);
          if (a) mine[on + __popc(m & ((1u << lane) - 1))] = static_cast<unsigned short>(i);
          on += __popc(m);
        }
        n = on;
        if (!kShort && lane == 0) listed = on;
      }
      if constexpr (kShort) {
        __syncwarp();
      } else {
        __syncthreads();
        n = listed;
      }
    }
    auto row_at = [&](int k) -> long long {
      return first + (base + (masked ? mine[k] : k)) * step;
    };
    auto issue = [&](int k) {
      const int e = k * abreast + sub;
      if (e < n) {
        const long long off = row_at(e) * p.H;
        uint4* slot = ring + static_cast<size_t>(k % kStages) * arrays * NV * cta + tid;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (j * blockDim.x + threadIdx.x) * VEC;
          if (in[j]) {
            cp_async16(slot + j * cta, dy + off + c);
            cp_async16(slot + (NV + j) * cta, sv + off + c);
            if (with_ds) cp_async16(slot + (2 * NV + j) * cta, ds + off + c);
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
      const uint4* slot = ring + static_cast<size_t>(k % kStages) * arrays * NV * cta + tid;
      const int e = k * abreast + sub;
      const bool valid = !kShort || e < n;
      Raw<T, VEC> rdy[NV], rsv[NV];
      float ss = 0.f, gs = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (in[j] && valid) {
          rdy[j].v = slot[j * cta];
          rsv[j].v = slot[(NV + j) * cta];
          float s[VEC], d[VEC], wf[VEC];
          widen<T, VEC>(rsv[j], s);
          widen<T, VEC>(rdy[j], d);
          widen<T, VEC>(rw[j], wf);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            ss = fmaf(s[i], s[i], ss);
            gs = fmaf(d[i] * wf[i], s[i], gs);
          }
        }
      }
      if constexpr (kShort) {
        for (int o = blockDim.x / 2; o > 0; o /= 2) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          gs += __shfl_xor_sync(0xffffffffu, gs, o);
        }
      } else {
        reduce_pair<false>(ss, gs, red[parity], blockDim.x >> 5);
        parity ^= 1;
      }
      if (!valid) continue;
      const float rstd = rsqrtf(fmaf(ss, inv_h, p.eps));
      const float c2 = gs * rstd * rstd * inv_h;
      const long long off = row_at(e) * p.H;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (in[j]) {
          const int c = (j * blockDim.x + threadIdx.x) * VEC;
          float s[VEC], d[VEC], wf[VEC], o[VEC] = {};
          widen<T, VEC>(rsv[j], s);
          widen<T, VEC>(rdy[j], d);
          widen<T, VEC>(rw[j], wf);
          if (with_ds) {
            Raw<T, VEC> r;
            r.v = slot[(2 * NV + j) * cta];
            widen<T, VEC>(r, o);
          }
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            o[i] = fmaf(rstd, fmaf(-s[i], c2, d[i] * wf[i]), o[i]);
            acc[j][i] = fmaf(d[i], s[i] * rstd, acc[j][i]);
          }
          store_vec<T, VEC>(dx + off + c, o);
        }
      }
    }
    cp_async_wait<0>();
    // the list is written again only after every warp is done with it
    if (masked && base + kListRows < rows) {
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
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        for (int o = blockDim.x; o < 32; o *= 2) acc[j][i] += __shfl_xor_sync(0xffffffffu, acc[j][i], o);
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (in[j] && sub == 0) {
#pragma unroll
        for (int h = 0; h < VEC; h += 4)
          *reinterpret_cast<float4*>(sums + warp * p.H + c + h) =
              make_float4(acc[j][h], acc[j][h + 1], acc[j][h + 2], acc[j][h + 3]);
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
      const int c = (j * blockDim.x + threadIdx.x) * VEC;
      if (in[j]) {
#pragma unroll
        for (int h = 0; h < VEC; h += 4)
          *reinterpret_cast<float4*>(out + c + h) =
              make_float4(acc[j][h], acc[j][h + 1], acc[j][h + 2], acc[j][h + 3]);
      }
    }
  }
}

// dx = ds or 0 on the inactive rows, for the ring kernel; it runs beside that
// one.  Small CTAs in the order of the rows: where the ring kernel's CTAs wrote
// these rows themselves, one a SM and each at its own pace, [131072, 7168] bf16
// with 10 % active rows took 388 us against 350.
struct FillArgs {
  const uint4* ds;        // or null
  uint4* dx;
  const uint8_t* mask;
  long long R;
  int vecs;               // 16-byte vectors of a row
  int rows;               // rows of a CTA
};
__global__ void __launch_bounds__(256) norm_bwd_fill_kernel(const FillArgs p) {
  const long long r0 = static_cast<long long>(blockIdx.x) * p.rows;
  for (int r = threadIdx.y; r < p.rows && r0 + r < p.R; r += blockDim.y) {
    if (p.mask[r0 + r] != 0) continue;
    const long long off = (r0 + r) * p.vecs;
#pragma unroll 4
    for (int v = threadIdx.x; v < p.vecs; v += blockDim.x)
      p.dx[off + v] = p.ds ? p.ds[off + v] : make_uint4(0, 0, 0, 0);
  }
  wait_for_launch_before();   // whoever waits for this launch waits for the ring kernel too
}

// Rows too long for registers: dx in two walks of the row, the row's rstd
// kept for the dw pass.
template <typename T>
__global__ void __launch_bounds__(1024)
rmsnorm_bwd_long_kernel(const RmsNormBwdArgs p) {
  __shared__ float2 red[32];
  const long long row = blockIdx.x;
  const T* dy = static_cast<const T*>(p.dy) + row * p.H;
  const T* sp = static_cast<const T*>(p.s) + row * p.H;
  const T* w = static_cast<const T*>(p.w);
  const T* ds = p.ds ? static_cast<const T*>(p.ds) + row * p.H : nullptr;
  T* dx = static_cast<T*>(p.dx) + row * p.H;
  const bool active = !p.mask || p.mask[row] != 0;
  float ss = 0.f, gs = 0.f;
  if (active) {
    for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
      const float s = to_f32(sp[c]);
      ss = fmaf(s, s, ss);
      gs = fmaf(to_f32(dy[c]) * to_f32(w[c]), s, gs);
    }
    reduce_pair<false>(ss, gs, red, blockDim.x >> 5);
  }
  const float inv_h = 1.f / static_cast<float>(p.H);
  const float rstd = rsqrtf(fmaf(ss, inv_h, p.eps));
  const float c2 = gs * rstd * rstd * inv_h;
  for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
    float o[1] = {ds ? to_f32(ds[c]) : 0.f};
    if (active) o[0] = fmaf(rstd, fmaf(-to_f32(sp[c]), c2, to_f32(dy[c]) * to_f32(w[c])), o[0]);
    store_vec<T, 1>(dx + c, o);
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
rmsnorm_dw_kernel(const float* __restrict__ partial, int n, int H, float* __restrict__ dw) {
  __shared__ float sm[kDwWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.f;
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

struct RowShape {
  int vec;       // elements of a vector: 16 bytes where every row is aligned, else 1
  int nv;        // vectors a thread: 1, 2, 4 or 8; 0: too long for registers
  int threads;   // threads of a row, a multiple of 32
  int rows;      // rows of a CTA (> 1 only where a warp holds a row)
};

// A row of H elements in registers.  Aligned rows: the fewest vectors a thread
// that 1024 threads allow.  Element by element: up to eight a thread before a
// CTA grows beyond 256 threads, so that several rows share an SM.  Rows that a
// warp can hold share a CTA, one warp each.
RowShape row_shape(int H, int vec16) {
  RowShape s;
  s.vec = H % vec16 == 0 ? vec16 : 1;
  const int n = (H + s.vec - 1) / s.vec;
  const int wide = s.vec == 1 ? 256 : 1024;
  s.nv = 1;
  while (s.nv < 8 && n > wide * s.nv) s.nv *= 2;
  if (n > 1024 * s.nv) return {s.vec, 0, 1024, 1};
  s.threads = ((n + s.nv - 1) / s.nv + 31) / 32 * 32;
  s.rows = s.threads == 32 ? 4 : 1;
  return s;
}

}  // namespace

// Partial rows of dw that rmsnorm_bwd writes at most, for any machine size (a
// CTA of short rows writes eight).
long long rmsnorm_bwd_partials(long long R, long long H) {
  const long long most = H <= 32768 ? 1024 : 32;
  return R < 8 ? 8 : R < most ? R : most;
}

template <typename T, int VEC>
static cudaError_t fwd_nv(const RmsNormFwdArgs& a, const RowShape& sh, cudaStream_t s) {
  const dim3 block(sh.threads, sh.rows);
  const unsigned grid = static_cast<unsigned>((a.R + sh.rows - 1) / sh.rows);
  switch (sh.nv) {
    case 1: rmsnorm_fwd_kernel<T, VEC, 1><<<grid, block, 0, s>>>(a); break;
    case 2: rmsnorm_fwd_kernel<T, VEC, 2><<<grid, block, 0, s>>>(a); break;
    case 4: rmsnorm_fwd_kernel<T, VEC, 4><<<grid, block, 0, s>>>(a); break;
    default: rmsnorm_fwd_kernel<T, VEC, 8><<<grid, block, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

template <typename T>
static cudaError_t fwd_t(const RmsNormFwdArgs& a, cudaStream_t s) {
  const RowShape sh = row_shape(a.H, kVec16<T>);
  if (sh.nv == 0) {
    rmsnorm_fwd_long_kernel<T><<<static_cast<unsigned>(a.R), 1024, 0, s>>>(a);
    return cudaGetLastError();
  }
  return sh.vec == 1 ? fwd_nv<T, 1>(a, sh, s) : fwd_nv<T, kVec16<T>>(a, sh, s);
}

cudaError_t launch_rmsnorm_fwd(const RmsNormFwdArgs& a, int is_bf16, cudaStream_t s) {
  if (a.R == 0) return cudaSuccess;
  return is_bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

template <typename T, int VEC>
static cudaError_t bwd_nv(const RmsNormBwdArgs& a, const RowShape& sh, unsigned grid,
                          cudaStream_t s) {
  const dim3 block(sh.threads, sh.rows);
  if constexpr (VEC == 1) {
    if (sh.nv == 1) rmsnorm_bwd_kernel<T, VEC, 1><<<grid, block, 0, s>>>(a);
    else if (sh.nv == 2) rmsnorm_bwd_kernel<T, VEC, 2><<<grid, block, 0, s>>>(a);
  }
  if (sh.nv == 4) rmsnorm_bwd_kernel<T, VEC, 4><<<grid, block, 0, s>>>(a);
  else if (sh.nv == 8) rmsnorm_bwd_kernel<T, VEC, 8><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}

// The ring kernel's shape for rows of H elements that start on 16-byte
// boundaries; stages 0: none (longer rows).
// About 512 threads an SM, two or four vectors each: at [65536, 8192] bf16 with
// ds, one row by 1024 threads of one vector took 742 us, by 512 of two 600.
// Three rows deep: 600 us against 630 with two and 639 with four; at
// [65536, 4096] fp32 477 against 508 and 525.  Short rows, two CTAs an SM (room
// for 128 registers) against three: [524288, 128] bf16 68 us against 81.
struct RingShape {
  int nv, lanes, groups;   // block (lanes, groups); groups > 1: rows within warps
  int ctas, stages;
  size_t smem;
};

RingShape ring_shape(int H, int vec16, int arrays) {
  RingShape r = {};
  const int n = H / vec16;
  if (H % vec16 != 0 || n > 2048) return r;
  if (n <= 128) {
    r.nv = n <= 64 ? 2 : 4;
    r.lanes = n <= 16 ? 8 : n <= 32 ? 16 : 32;
    r.groups = 32 * kShortWarps / r.lanes;
  } else {
    r.nv = n <= 1024 ? 2 : 4;
    r.lanes = ((n + r.nv - 1) / r.nv + 31) / 32 * 32;
    r.groups = 1;
  }
  const int cta = r.lanes * r.groups;
  r.ctas = cta < 512 ? 512 / cta : 1;
  const size_t stage = static_cast<size_t>(arrays) * r.nv * cta * 16;
  r.stages = r.ctas * 3 * stage <= 200u << 10 ? 3 : 2;
  r.smem = r.stages * stage;
  return r;
}

template <typename T, int NV, int S, bool kShort, bool kDs, bool kMask>
static cudaError_t ring_launch(const RmsNormBwdArgs& a, const RingShape& r, unsigned grid,
                               cudaStream_t s) {
  const auto kernel = rmsnorm_bwd_ring_kernel<T, NV, S, kShort, kDs, kMask>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(r.smem));
  if (e != cudaSuccess) return e;
  kernel<<<grid, dim3(r.lanes, r.groups), r.smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int NV, int S>
static cudaError_t ring_kind(const RmsNormBwdArgs& a, const RingShape& r, unsigned grid,
                             cudaStream_t s) {
  if (r.groups > 1) return ring_launch<T, NV, S, true, false, false>(a, r, grid, s);
  if (a.ds)
    return a.mask ? ring_launch<T, NV, S, false, true, true>(a, r, grid, s)
                  : ring_launch<T, NV, S, false, true, false>(a, r, grid, s);
  return a.mask ? ring_launch<T, NV, S, false, false, true>(a, r, grid, s)
                : ring_launch<T, NV, S, false, false, false>(a, r, grid, s);
}

template <typename T>
static cudaError_t ring_run(const RmsNormBwdArgs& a, const RingShape& r, unsigned grid,
                            cudaStream_t s) {
  if (r.nv == 2)
    return r.stages == 2 ? ring_kind<T, 2, 2>(a, r, grid, s) : ring_kind<T, 2, 3>(a, r, grid, s);
  return r.stages == 2 ? ring_kind<T, 4, 2>(a, r, grid, s) : ring_kind<T, 4, 3>(a, r, grid, s);
}

template <typename T>
static cudaError_t bwd_t(const RmsNormBwdArgs& a, int num_sms, int* n_partials, cudaStream_t s) {
  const RowShape sh = row_shape(a.H, kVec16<T>);
  const long long most = rmsnorm_bwd_partials(a.R, a.H);
  const RingShape ring = ring_shape(a.H, kVec16<T>, a.ds ? 3 : 2);
  if (ring.stages > 0) {
    const int abreast = ring.groups > 1 ? kShortWarps : 1;
    long long grid = static_cast<long long>(num_sms) * ring.ctas;
    const long long need = (a.R + abreast - 1) / abreast;
    if (grid > need) grid = need > 0 ? need : 1;
    if (grid > most) grid = most;
    *n_partials = static_cast<int>(grid);
    const cudaError_t e = ring_run<T>(a, ring, static_cast<unsigned>(grid), s);
    if (e != cudaSuccess || !a.mask || a.ds == a.dx || a.R == 0) return e;   // in place: ds is there
    FillArgs f = {static_cast<const uint4*>(a.ds), static_cast<uint4*>(a.dx), a.mask, a.R,
                  a.H / kVec16<T>, 0};
    f.rows = f.vecs >= 4096 ? 1 : 4096 / f.vecs < 256 ? 4096 / f.vecs : 256;   // about 64 KB
    int tx = 16;
    while (tx < 256 && tx < f.vecs) tx *= 2;
    const long long fill = (a.R + f.rows - 1) / f.rows;
    return launch_overlapped(norm_bwd_fill_kernel, dim3(static_cast<unsigned>(fill)),
                             dim3(tx, 256 / tx), 0, s, f);
  }
  if (sh.nv == 0) {
    const int splits = static_cast<int>(most < 32 ? most : 32);
    if (a.R > 0) rmsnorm_bwd_long_kernel<T><<<static_cast<unsigned>(a.R), 1024, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    rmsnorm_dw_long_kernel<T><<<dim3((a.H + 255) / 256, splits), 256, 0, s>>>(a);
    *n_partials = splits;
    return cudaGetLastError();
  }
  // resident CTAs: 2048 threads an SM, at most one row a CTA left over
  int per_sm = 2048 / (sh.threads * sh.rows);
  if (per_sm > 4) per_sm = 4;
  long long grid = static_cast<long long>(num_sms) * per_sm;
  const long long need = (a.R + sh.rows - 1) / sh.rows;
  if (grid > need) grid = need;
  if (grid * sh.rows > most) grid = most / sh.rows;
  if (grid < 1) grid = 1;
  *n_partials = static_cast<int>(grid * sh.rows);
  return sh.vec == 1 ? bwd_nv<T, 1>(a, sh, static_cast<unsigned>(grid), s)
                     : bwd_nv<T, kVec16<T>>(a, sh, static_cast<unsigned>(grid), s);
}

cudaError_t launch_rmsnorm_bwd(const RmsNormBwdArgs& a, int is_bf16, int num_sms, int* n_partials,
                               cudaStream_t s) {
  return is_bf16 ? bwd_t<__nv_bfloat16>(a, num_sms, n_partials, s)
                 : bwd_t<float>(a, num_sms, n_partials, s);
}

cudaError_t launch_rmsnorm_dw(const float* partial, int n, int H, float* dw, cudaStream_t s) {
  rmsnorm_dw_kernel<<<(H + 31) / 32, 32 * kDwWarps, 0, s>>>(partial, n, H, dw);
  return cudaGetLastError();
}

}  // namespace eas
