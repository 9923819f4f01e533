// Scores of logits that exist: log probabilities of given tokens, entropy, the top
// alternatives of each row, and the gradient of all of them at the logits.
//
// With c = scale log2 e, a row's statistics are kept in base 2:
//   m = max x,  y = c (x - m),  s = sum 2^y,  u = sum 2^y y,
//   lse = scale m + ln s,  logp(t) = scale (x_t - m) - ln s,  H = ln s - ln2 u / s.
// x - m comes before the product, so values near the type's largest do not overflow.
// A value is read once; each thread keeps (m, s, u) of what it has seen and
// rescales s and u when a group of its values has a larger m.
//
// The k largest values come from the same pass.  The thread maxima are maxima of
// disjoint parts of the row, so t, the k-th largest of them, is no larger than the
// k-th largest value, and only parts whose maximum reaches t hold values that can be
// among the k: about k of 512 parts are read again (from L2), and what reaches t
// there is ordered.  Order is by (value, then lower column), kept in 64 bits:
// monotonic value bits above the complement of the column.
//
// Backward, with G = sum of a row's g_j and p = 2^(c x - log2 e lse):
//   dx_v = scale (sum_j g_j [v == t_j] - p_v (G + g_H (z_v - lse + H))).
#include "eas_device.cuh"
#include "eas_launch.cuh"
#include "eas_ops.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr int kThreads = 512;     // at most
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 4;         // vectors a thread loads at a time
constexpr int kCand = 1024;       // values above t that are kept
constexpr int kTies = 256;        // and values equal to it
constexpr int kTieParts = 96;     // parts whose maximum is t that are read again
constexpr int kMaxSplit = 8;      // CTAs a row
constexpr int kWhereScore = 40;   // `where` of the status word

// Row and column range of a CTA: vectors [v0, v1) of the row's 16-byte blocks, and,
// of the first and the last CTA of a row, the elements before and behind them.
template <typename T>
struct Slice {
  const T* row;
  int head, nvec, tail;      // of the whole row
  int v0, v1;
  bool first, last;
  __device__ Slice(const T* r, int V, int rank, int split) : row(r) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(r) & 15u) / static_cast<int>(sizeof(T));
    head = off ? kVec16<T> - off : 0;
    if (head > V) head = V;
    nvec = (V - head) / kVec16<T>;
    tail = V - head - nvec * kVec16<T>;
    const int per = (nvec + split - 1) / split;
    v0 = min(rank * per, nvec);
    v1 = min(v0 + per, nvec);
    first = rank == 0;
    last = rank == split - 1;
  }
  __device__ int column(int v) const { return head + v * kVec16<T>; }
  // Elements outside the vectors that this CTA has, and the i-th one's column.
  __device__ int loose() const { return (first ? head : 0) + (last ? tail : 0); }
  __device__ int loose_column(int i) const {
    if (first && i < head) return i;
    return head + nvec * kVec16<T> + i - (first ? head : 0);
  }
};

template <typename T>
__device__ __forceinline__ uint4 load_block(const T* row, int col) {
  return __ldg(reinterpret_cast<const uint4*>(row + col));
}

// A vector of -inf: what a thread takes where it has no vector left.
template <typename T>
__device__ __forceinline__ uint4 no_values() {
  const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  return make_uint4(w, w, w, w);
}

// Monotonic bits of a value: -0 as 0, NaN above everything; 0 stands for none.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0xffffffffu;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order_bits(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ unsigned long long order_key(uint32_t bits, int col) {
  return (static_cast<unsigned long long>(bits) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}

// ------------------------------------------------------------- statistics

struct Stats {
  float m, s, u;
};

// Exponents below this add nothing (2^-160 is 0 in fp32); values are raised to it
// so that -inf gives 0 * -160 and not 0 * -inf.
constexpr float kLeast = -160.f;

// Two statistics of one row.  s = 0: no value but -inf.  A NaN or +inf makes s NaN.
__device__ __forceinline__ Stats join(const Stats& a, const Stats& b, float c) {
  Stats r = {fmaxf(a.m, b.m), 0.f, 0.f};
  if (a.s != 0.f) {
    const float d = (a.m - r.m) * c, f = ex2_approx(d);
    r.s = f * a.s;
    r.u = f == 0.f ? 0.f : f * (a.u + d * a.s);
  }
  if (b.s != 0.f) {
    const float d = (b.m - r.m) * c, f = ex2_approx(d);
    r.s += f * b.s;
    r.u += f == 0.f ? 0.f : f * (b.u + d * b.s);
  }
  return r;
}

__device__ __forceinline__ void add_value(Stats& st, float x, float c) {
  const Stats one = {x, x == -INFINITY ? 0.f : x == INFINITY ? NAN : 1.f, 0.f};
  st = join(st, one, c);
}

// The larger of two values, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest of a group of vectors, NaN where one is.
template <typename T>
__device__ __forceinline__ float group_max(const uint4 (&r)[kGroup]) {
  if constexpr (sizeof(T) == 2) {
    auto h = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
    __nv_bfloat162 v = __hmax2_nan(h(r[0].x), h(r[0].y));
    v = __hmax2_nan(v, __hmax2_nan(h(r[0].z), h(r[0].w)));
#pragma unroll
    for (int i = 1; i < kGroup; ++i) {
      v = __hmax2_nan(v, __hmax2_nan(h(r[i].x), h(r[i].y)));
      v = __hmax2_nan(v, __hmax2_nan(h(r[i].z), h(r[i].w)));
    }
    return max_nan(__low2float(v), __high2float(v));
  } else {
    float v = -INFINITY;
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      v = max_nan(v, max_nan(max_nan(__uint_as_float(r[i].x), __uint_as_float(r[i].y)),
                             max_nan(__uint_as_float(r[i].z), __uint_as_float(r[i].w))));
    return v;
  }
}

// Two fp32 values in a register pair, as the packed instructions take them.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A thread's statistics while it walks: s and u in two halves.
struct Walk {
  float m = -INFINITY;
  f32x2 s = 0, u = 0;

  __device__ __forceinline__ void add_pair(float x0, float x1, f32x2 c2, f32x2 minus_m) {
    float y0, y1;
    unpack2(mul2(add2(pack2(x0, x1), minus_m), c2), y0, y1);
    y0 = fmaxf(y0, kLeast);
    y1 = fmaxf(y1, kLeast);
    const f32x2 e = pack2(ex2_approx(y0), ex2_approx(y1));
    s = add2(s, e);
    u = fma2(e, pack2(y0, y1), u);
  }

  template <typename T>
  __device__ __forceinline__ void add(const uint4 (&r)[kGroup], float c) {
    const float g = group_max<T>(r);
    if (!(g <= m)) {
      const float top = max_nan(m, g);
      if (m != -INFINITY) {
        const float d = fmaxf((m - top) * c, kLeast), f = ex2_approx(d);
        const f32x2 f2 = pack2(f, f);
        u = mul2(f2, fma2(pack2(d, d), s, u));
        s = mul2(f2, s);
      }
      m = top;
      if (!(top < INFINITY)) s = pack2(NAN, NAN);
    }
    const f32x2 c2 = pack2(c, c), minus_m = pack2(-m, -m);
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) add_pair(bf16_lo(w[j]), bf16_hi(w[j]), c2, minus_m);
      } else {
        add_pair(__uint_as_float(w[0]), __uint_as_float(w[1]), c2, minus_m);
        add_pair(__uint_as_float(w[2]), __uint_as_float(w[3]), c2, minus_m);
      }
    }
  }

  __device__ __forceinline__ Stats stats() const {
    float s0, s1, u0, u1;
    unpack2(s, s0, s1);
    unpack2(u, u0, u1);
    return {m, s0 + s1, u0 + u1};
  }
};

// ------------------------------------------------------------ the k largest

struct Shared {
  Stats warp[kWarps];
  Stats part[kMaxSplit];                          // of the row's CTAs, in CTA 0
  uint32_t best[kThreads];                        // order bits of the threads' maxima
  unsigned long long cand[kCand];
  unsigned long long tie[kTies];
  unsigned long long list[kMaxSplit * kMaxTop];   // the CTAs' k largest, in CTA 0
  int scan[kWarps];
  uint32_t t;
  int n_above, n_tie, total;
};

// Order bits of the 16-byte block's values.
template <typename T>
__device__ __forceinline__ void block_bits(const uint4& r, uint32_t (&b)[kVec16<T>]) {
  float f[kVec16<T>];
  Raw<T, kVec16<T>> raw;
  raw.v = r;
  widen<T, kVec16<T>>(raw, f);
#pragma unroll
  for (int j = 0; j < kVec16<T>; ++j) b[j] = order_bits(f[j]);
}

// The largest t such that k of the threads' maxima reach it (0: fewer have one).
// The bits below kLow are the same in every value of the type and its sign.
template <typename T>
__device__ __forceinline__ uint32_t kth_of_maxima(const uint32_t* best, int nt, int k, int lane) {
  constexpr int kLow = sizeof(T) == 2 ? 16 : 0;
  uint32_t key[kWarps];
#pragma unroll
  for (int i = 0; i < kWarps; ++i) key[i] = i * 32 < nt ? best[i * 32 + lane] : 0u;
  uint32_t t = 0;
#pragma unroll 1
  for (int bit = 31; bit >= kLow; --bit) {
    const uint32_t c = t | (1u << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) n += key[i] >= c;
    if (__reduce_add_sync(0xffffffffu, n) >= k) t = c;
  }
  // a negative value's low bits are ones
  if (kLow && t && !(t & 0x80000000u)) t |= (1u << kLow) - 1;
  return t;
}

// Sum over the CTA of a count, and what the threads before this one have of it.
__device__ __forceinline__ int scan_counts(int n, int* scan, int nt, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  return before + inc - n;
}

// The first `need` values equal to t of the slice, by column, to sm.cand[from ..].
template <typename T>
__device__ void first_ties(const Slice<T>& sl, Shared& sm, uint32_t t, int from, int need) {
  constexpr int VEC = kVec16<T>;
  const int nt = blockDim.x, tid = threadIdx.x;
  int have = 0;
  // head, blocks of nt vectors, tail
  const int steps = (sl.v1 - sl.v0 + nt - 1) / nt;
#pragma unroll 1
  for (int i = -1; i <= steps && have < need; ++i) {
    uint32_t b[VEC] = {};
    int col = 0, count = 0;
    if (i < 0 || i == steps) {
      const int n = i < 0 ? (sl.first ? sl.head : 0) : (sl.last ? sl.tail : 0);
      if (tid < n) {
        col = i < 0 ? tid : sl.head + sl.nvec * VEC + tid;
        b[0] = order_bits(to_f32(sl.row[col]));
      }
    } else {
      const int v = sl.v0 + i * nt + tid;
      if (v < sl.v1) {
        col = sl.column(v);
        block_bits<T>(load_block(sl.row, col), b);
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) count += b[j] == t;
    int total;
    int at = have + scan_counts(count, sm.scan, nt, total);
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (b[j] == t) {
        if (at < need) sm.cand[from + at] = order_key(t, col + j);
        ++at;
      }
    have += total;
  }
  __syncthreads();
}

// Calls f(order bits, column) for every value of the slice.
template <typename T, typename F>
__device__ __forceinline__ void for_all(const Slice<T>& sl, F f) {
  constexpr int VEC = kVec16<T>;
  for (int v = sl.v0 + threadIdx.x; v < sl.v1; v += blockDim.x) {
    uint32_t b[VEC];
    const int col = sl.column(v);
    block_bits<T>(load_block(sl.row, col), b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f(b[j], col + j);
  }
  if (static_cast<int>(threadIdx.x) < sl.loose()) {
    const int col = sl.loose_column(threadIdx.x);
    f(order_bits(to_f32(sl.row[col])), col);
  }
}

__device__ __forceinline__ void push(unsigned long long* list, int* n, int most, uint32_t b, int col) {
  const int at = atomicAdd(n, 1);
  if (at < most) list[at] = order_key(b, col);
}

// The k largest of the slice in order, to `out` (0 where it has fewer).  `best`:
// order bits of this thread's maximum over its vectors, 0 if it has none.
template <typename T>
__device__ void k_largest(const Slice<T>& sl, Shared& sm, uint32_t best, int k,
                          unsigned long long* out) {
  constexpr int VEC = kVec16<T>;
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sm.best[tid] = best;
  if (tid == 0) sm.n_above = sm.n_tie = 0;
  __syncthreads();
  if (warp == 0) {
    const uint32_t t = kth_of_maxima<T>(sm.best, nt, k, lane);
    if (lane == 0) sm.t = t;
  }
  __syncthreads();
  uint32_t t = sm.t;
  // many parts with the same maximum (a row of equal values, or of -inf): their ties
  // are looked for in the order of the columns instead
  const bool take_ties = t != 0 && __syncthreads_count(best == t) <= kTieParts;
  unsigned parts = __ballot_sync(0xffffffffu, best > t || (take_ties && best == t));
  while (parts) {
    const int owner = __ffs(parts) - 1;
    parts &= parts - 1;
    for (int v = sl.v0 + warp * 32 + owner + lane * nt; v < sl.v1; v += 32 * nt) {
      uint32_t b[VEC];
      const int col = sl.column(v);
      block_bits<T>(load_block(sl.row, col), b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (b[j] > t) push(sm.cand, &sm.n_above, kCand, b[j], col + j);
        else if (take_ties && b[j] == t) push(sm.tie, &sm.n_tie, kTies, b[j], col + j);
      }
    }
  }
  if (tid < sl.loose()) {
    const int col = sl.loose_column(tid);
    const uint32_t b = order_bits(to_f32(sl.row[col]));
    if (b > t) push(sm.cand, &sm.n_above, kCand, b, col);
    else if (take_ties && b == t) push(sm.tie, &sm.n_tie, kTies, b, col);
  }
  __syncthreads();
  int n = sm.n_above;
  const int ties = sm.n_tie;
  bool look = t != 0 && n < k && !(take_ties && ties <= kTies);
  if (n > kCand) {
    // the few parts that reach t hold too many values above it (a row whose values
    // lie in the order of its parts): the k-th largest value itself, bit by bit
    t = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = t | (1u << bit);
      int count = 0, total;
      for_all(sl, [&](uint32_t b, int) { count += b >= c; });
      scan_counts(count, sm.scan, nt, total);
      if (total >= k) t = c;
    }
    __syncthreads();
    if (tid == 0) sm.n_above = 0;
    __syncthreads();
    for_all(sl, [&](uint32_t b, int col) {
      if (b > t) push(sm.cand, &sm.n_above, kCand, b, col);
    });
    __syncthreads();
    n = sm.n_above;               // below k
    look = true;
  }
  if (look) {
    first_ties(sl, sm, t, n, k - n);
    n = k;
  } else if (n < k && t != 0) {
    for (int i = tid; i < ties; i += nt) sm.cand[n + i] = sm.tie[i];
    n += ties;
    __syncthreads();
  }
  // their places by counting
  for (int i = tid; i < n; i += nt) {
    const unsigned long long key = sm.cand[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += sm.cand[j] > key;
    if (place < k) out[place] = key;
  }
  for (int i = n + tid; i < k; i += nt) out[i] = 0;
}

// ------------------------------------------------------------------ cluster

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta0(const void* p) {
  uint32_t out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(out) : "r"(smem_u32(p)));
  return out;
}
__device__ __forceinline__ void store_cta0(const unsigned long long* p, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_cta0(p)), "l"(v) : "memory");
}
__device__ __forceinline__ void store_cta0(const float* p, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(in_cta0(p)), "f"(v) : "memory");
}

// A row a cluster of a.split CTAs (1: no cluster).
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) score_fwd_kernel(const ScoreFwdArgs a) {
  __shared__ Shared sm;
  const int split = a.split, rank = split > 1 ? blockIdx.x % split : 0;
  const long long row = blockIdx.x / split;
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (a.mask && !a.mask[row]) {
    if (rank == 0) {
      for (int j = tid; j < a.M; j += nt) a.logprob[row * a.M + j] = 0.f;
      for (int j = tid; j < a.k; j += nt) {
        a.top[row * a.k + j] = 0.f;
        a.ids[row * a.k + j] = -1;
      }
      if (tid == 0) a.entropy[row] = a.lse[row] = 0.f;
    }
    return;
  }
  if (split > 1) cluster_arrive();         // CTA 0 is there before it is written to
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  const Slice<T> sl(x, a.V, rank, split);

  Walk w;
  for (int v = sl.v0 + tid; v < sl.v1; v += kGroup * nt) {
    uint4 r[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      r[i] = v + i * nt < sl.v1 ? load_block(x, sl.column(v + i * nt)) : no_values<T>();
    w.add<T>(r, a.c);
  }
  const uint32_t best = sl.v0 + tid < sl.v1 ? order_bits(w.m) : 0u;
  Stats st = w.stats();
  if (tid < sl.loose()) add_value(st, to_f32(x[sl.loose_column(tid)]), a.c);
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    Stats o;
    o.m = __shfl_xor_sync(0xffffffffu, st.m, d);
    o.s = __shfl_xor_sync(0xffffffffu, st.s, d);
    o.u = __shfl_xor_sync(0xffffffffu, st.u, d);
    st = lane & d ? join(o, st, a.c) : join(st, o, a.c);
  }
  if (lane == 0) sm.warp[warp] = st;
  if (a.k) k_largest(sl, sm, best, a.k, sm.list);
  __syncthreads();
  if (tid == 0) {
    st = sm.warp[0];
    for (int i = 1; i < nt / 32; ++i) st = join(st, sm.warp[i], a.c);
    sm.part[0] = st;
  }
  if (split > 1) {
    __syncthreads();
    cluster_wait();
    if (rank) {
      for (int i = tid; i < a.k; i += nt) store_cta0(&sm.list[rank * a.k + i], sm.list[i]);
      if (tid == 0) {
        store_cta0(&sm.part[rank].m, st.m);
        store_cta0(&sm.part[rank].s, st.s);
        store_cta0(&sm.part[rank].u, st.u);
      }
    }
    cluster_arrive();
    cluster_wait();
    if (rank) return;
    st = sm.part[0];
    for (int i = 1; i < split; ++i) st = join(st, sm.part[i], a.c);
    // a value's place: its own in its list and how many of each other list are larger
    for (int i = tid; i < split * a.k; i += nt) {
      const unsigned long long key = sm.list[i];
      const int own = i / a.k;
      int place = i - own * a.k;
      for (int o = 0; o < split; ++o) {
        if (o == own) continue;
        int lo = 0, hi = a.k;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (sm.list[o * a.k + mid] > key) lo = mid + 1;
          else hi = mid;
        }
        place += lo;
      }
      if (key && place < a.k) sm.cand[place] = key;
    }
    __syncthreads();
  } else {
    __syncthreads();
    st = sm.part[0];
  }

  const unsigned long long* sorted = split > 1 ? sm.cand : sm.list;
  const float ls = st.s > 0.f ? logf(st.s) : NAN;      // no finite value: NaN
  for (int j = tid; j < a.k; j += nt) {
    const unsigned long long key = sorted[j];
    a.top[row * a.k + j] = fmaf(from_order_bits(static_cast<uint32_t>(key >> 32)) - st.m, a.scale, -ls);
    a.ids[row * a.k + j] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
  }
  for (int j = tid; j < a.M; j += nt) {
    const int t = a.tokens[row * a.M + j];
    float lp = 0.f;
    if (t >= 0 && t < a.V) lp = fmaf(to_f32(x[t]) - st.m, a.scale, -ls);
    else if (t != -1 && a.status) report(a.status, kStInvalidArg, kWhereScore, static_cast<int>(row));
    a.logprob[row * a.M + j] = lp;
  }
  if (tid == 0) {
    a.lse[row] = fmaf(st.m, a.scale, ls);
    a.entropy[row] = ls - kLn2 * (st.u / st.s);
  }
}

// ----------------------------------------------------------------- backward

// blockIdx.x = row * split + part of the row.
template <typename T>
__global__ void __launch_bounds__(kThreads) score_bwd_kernel(const ScoreBwdArgs a) {
  constexpr int VEC = kVec16<T>;
  __shared__ int tok[kMaxTokens];
  __shared__ float g[kMaxTokens];
  __shared__ float sum;
  const int split = a.split, rank = blockIdx.x % split;
  const long long row = blockIdx.x / split;
  const int nt = blockDim.x, tid = threadIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
  const Slice<T> sl(x, a.V, rank, split);
  const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) & 15u) == 0;
  const bool on = !a.mask || a.mask[row];

  float c0 = 0.f, c1 = 0.f, lse = 0.f;    // -scale p (G + g_H (d + H)) = p (c0 + c1 d), d = z - lse
  if (on) {
    for (int j = tid; j < a.M; j += nt) {
      const int t = a.tokens[row * a.M + j];
      const bool real = t >= 0 && t < a.V;
      if (!real && t != -1 && a.status) report(a.status, kStInvalidArg, kWhereScore, static_cast<int>(row));
      tok[j] = real ? t : -1;
      g[j] = real ? a.g_logprob[row * a.M + j] : 0.f;
    }
    __syncthreads();
    if (tid < 32) {
      float s = 0.f;
      for (int j = tid; j < a.M; j += 32) s += g[j];
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (tid == 0) sum = s;
    }
    __syncthreads();
    const float gh = a.g_entropy ? a.g_entropy[row] : 0.f;
    lse = a.lse[row];
    c0 = -a.scale * (sum + gh * a.entropy[row]);
    c1 = -a.scale * gh;
  }
  auto value = [&](float xv) {
    const float d = max_nan(fmaf(xv, a.scale, -lse), kLeast);
    return ex2_approx(d * kLog2e) * fmaf(c1, d, c0);
  };
  // the values at the given tokens, before dx (which may be x) is written
  float at_token = 0.f;
  bool mine = false;
  if (on && tid < a.M && tok[tid] >= 0) {
    const int t = tok[tid], v = (t - sl.head) / VEC;
    const bool vec = t >= sl.head && v < sl.nvec;
    mine = vec ? v >= sl.v0 && v < sl.v1 : t < sl.head ? sl.first : sl.last;
    float s = 0.f;
    for (int j = 0; j < a.M; ++j)
      if (tok[j] == t) {
        if (j < tid) mine = false;       // the token's first entry writes
        s += g[j];
      }
    if (mine) at_token = fmaf(a.scale, s, value(to_f32(x[t])));
  }
  __syncthreads();
  if (tid < sl.loose()) {
    const int col = sl.loose_column(tid);
    const float d[1] = {on ? value(to_f32(x[col])) : 0.f};
    store_vec<T, 1>(dx + col, d);
  }
  constexpr int kUnroll = 4;
  for (int v = sl.v0 + tid; v < sl.v1; v += kUnroll * nt) {
    Raw<T, VEC> r[kUnroll];
    if (on) {
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
        if (v + i * nt < sl.v1) r[i] = load_raw<T, VEC>(x + sl.column(v + i * nt));
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (v + i * nt >= sl.v1) break;
      const int col = sl.column(v + i * nt);
      float f[VEC] = {};
      if (on) {
        widen<T, VEC>(r[i], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = value(f[j]);
      }
      if (same) {
        store_vec<T, VEC, true>(dx + col, f);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d[1] = {f[j]};
          store_vec<T, 1>(dx + col + j, d);
        }
      }
    }
  }
  __syncthreads();
  if (mine) {
    const float d[1] = {at_token};
    store_vec<T, 1>(dx + tok[tid], d);
  }
}

// Threads a row: about two groups of loads each, so that short rows do not leave
// most of a CTA idle.
int threads_of(long long nvec) {
  int nt = kThreads;
  while (nt > 64 && nvec < 2 * nt) nt >>= 1;
  return nt;
}

}  // namespace

cudaError_t launch_score_fwd(const ScoreFwdArgs& args, int is_bf16, int num_sms, cudaStream_t s) {
  if (args.N == 0) return cudaSuccess;
  ScoreFwdArgs a = args;
  const long long nvec = a.V / (is_bf16 ? 8 : 4);
  const int nt = threads_of(nvec);
  // few rows: each by several CTAs, until the machine has two CTAs an SM or a thread
  // a vector
  a.split = 1;
  while (a.split < kMaxSplit && a.N * a.split * 2 <= 2LL * num_sms && nvec >= 2LL * a.split * nt) a.split *= 2;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(a.split), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.N * a.split));
  cfg.blockDim = dim3(nt);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = a.split > 1 ? 1 : 0;
  return is_bf16 ? cudaLaunchKernelEx(&cfg, score_fwd_kernel<__nv_bfloat16>, a)
                 : cudaLaunchKernelEx(&cfg, score_fwd_kernel<float>, a);
}

cudaError_t launch_score_bwd(const ScoreBwdArgs& args, int is_bf16, int num_sms, cudaStream_t s) {
  if (args.N == 0) return cudaSuccess;
  ScoreBwdArgs a = args;
  const long long nvec = a.V / (is_bf16 ? 8 : 4);
  int nt = threads_of(nvec);
  if (nt < kMaxTokens && a.M > nt) nt = kMaxTokens;
  a.split = 1;
  while (a.split < 64 && a.N * a.split * 2 <= 4LL * num_sms && nvec >= 2LL * a.split * nt) a.split *= 2;
  const dim3 grid(static_cast<unsigned>(a.N * a.split));
  if (is_bf16) score_bwd_kernel<__nv_bfloat16><<<grid, nt, 0, s>>>(a);
  else score_bwd_kernel<float><<<grid, nt, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace eas
