// Typed vector access shared by the elementwise and row kernels: VEC
// consecutive elements of T as one load or store, widened to fp32 registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace eas {

// Elements of T in a 16-byte vector.
template <typename T>
constexpr int kVec16 = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// One vector of VEC elements as loaded, before widening.
template <typename T, int VEC>
struct Raw;
template <typename T>
struct Raw<T, 1> {
  T v;
};
template <>
struct Raw<float, 4> {
  uint4 v;
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 v;
};

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1)
    r.v = *p;
  else
    r.v = *reinterpret_cast<const uint4*>(p);
  return r;
}

// The same from memory that neither the kernel nor an overlapped launch before it
// writes: the load may move ahead of stores and waits.
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_const(const T* p) {
  Raw<T, VEC> r;
  if constexpr (VEC == 1)
    r.v = __ldg(p);
  else
    r.v = __ldg(reinterpret_cast<const uint4*>(p));
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void widen(const Raw<T, VEC>& r, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_f32(r.v);
  } else if constexpr (sizeof(T) == 4) {
    f[0] = __uint_as_float(r.v.x);
    f[1] = __uint_as_float(r.v.y);
    f[2] = __uint_as_float(r.v.z);
    f[3] = __uint_as_float(r.v.w);
  } else {
    f[0] = bf16_lo(r.v.x); f[1] = bf16_hi(r.v.x);
    f[2] = bf16_lo(r.v.y); f[3] = bf16_hi(r.v.y);
    f[4] = bf16_lo(r.v.z); f[5] = bf16_hi(r.v.z);
    f[6] = bf16_lo(r.v.w); f[7] = bf16_hi(r.v.w);
  }
}

// Rounds to T (nearest-even) and stores VEC consecutive elements.  kStream: they
// are the first to leave L2.
template <typename T, int VEC, bool kStream = false>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (sizeof(T) == 4)
      *p = f[0];
    else
      *p = __float2bfloat16_rn(f[0]);
  } else {
    uint4 u;
    if constexpr (sizeof(T) == 4) {
      u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]));
    } else {
      u = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                     pack_bf16x2(f[6], f[7]));
    }
    if constexpr (kStream)
      __stcs(reinterpret_cast<uint4*>(p), u);
    else
      *reinterpret_cast<uint4*>(p) = u;
  }
}

}  // namespace eas
