// Scores of logits that exist: log probabilities of given tokens, entropy, the top
// alternatives of each row, and the gradient of all of them at the logits.
//
// With c = scale log2 e, a row's statistics are kept in base 2:
//   y = c x - fp32(c m),  s = sum 2^y,  u = sum 2^y y,
//   lse = scale m + ln2 (log2 s - (c m - fp32(c m))),
//   logp(t) = ln2 (y_t - log2 s),
//   H = ln2 (log2 s - u / s),
// (where c m is so large that its rounding would count, y = c (x - m) and c m itself below),
// m being close to the largest x: a value is read once, each thread keeps (m, s, u) of
// what it has seen and moves m when a group of its values reaches 2^4 beyond it (a
// larger step would cost digits of y).
//
// The k largest values come from the same pass.  The thread maxima are maxima of
// disjoint parts of the row, so t, the k-th largest of them, is no larger than the
// k-th largest value.  Each thread also keeps the maxima of (up to 8) pieces of its
// part; only pieces whose maximum reaches t can hold values that are among the k, about
// k pieces of a few dozen values: those are read again (from L2), and what reaches t
// there is ordered.  Order is by (value, then lower column), kept in 64 bits:
// monotonic value bits above the complement of the column.
//
// Backward, with G = sum of a row's g_j and p = exp(z - lse), 1 at most (z - lse carries the
// rounding of an lse far from 0):
//   dx_v = scale (sum_j g_j [v == t_j] - p_v (G + g_H (z_v - lse + H))).
#include "eas_device.cuh"
#include "eas_launch.cuh"
#include "eas_ops.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr int kThreads = 512;     // at most
constexpr int kCand = 512;        // values that wait to be ordered
constexpr int kOrderAtOnce = 96;  // more are cut down first
constexpr int kPieces = 8;        // of a thread's part
constexpr int kTieThreads = 64;   // threads whose maximum is t, and
constexpr int kTiePieces = 256;   // pieces whose maximum is t that are read again, at most
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

// A vector that adds nothing to sums whose largest value is above kFillerMost, if c lies
// between kFillerLeast and kFillerScale (-1e30 everywhere, an exponent of -1e3 to -1e37):
// what a thread takes where it has none left.
constexpr float kFillerMost = -1e25f, kFillerLeast = 1e-27f, kFillerScale = 1e7f;
template <typename T>
__device__ __forceinline__ uint4 filler() {
  const uint32_t w = sizeof(T) == 2 ? 0xf14af14au : 0xf149f2cau;
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
// where -inf or the type's lowest values are among them, so that they give 0 * -160 and
// not 0 * -inf.
constexpr float kLeast = -160.f;

// Whether c m is far from 0: its rounding, part of every exponent below it, would be 2 or
// more, from 2^31 on beyond what 2^y takes.  NaN and infinities are far.
constexpr float kFar = 0x1p26f;
__device__ __forceinline__ bool is_far(float cm) { return !(fabsf(cm) <= kFar); }

// The exponent of x below m: c x - fp32(c m), or c (x - m).
__device__ __forceinline__ float exponent(float x, float m, float c) {
  const float cm = __fmul_rn(m, c);
  return is_far(cm) ? (x - m) * c : fmaf(x, c, -cm);
}
// What to add to an exponent below m to have one below n >= m.
__device__ __forceinline__ float shift(float m, float n, float c) {
  const float cm = __fmul_rn(m, c), cn = __fmul_rn(n, c);
  if (is_far(cn)) return is_far(cm) ? (m - n) * c : -fmaf(n, c, -cm);
  return is_far(cm) ? fmaf(m, c, -cn) : cm - cn;
}

// Two statistics of one row.  s = 0: no value but -inf.  A NaN or +inf makes s NaN.
__device__ __forceinline__ Stats join(const Stats& a, const Stats& b, float c) {
  Stats r = {fmaxf(a.m, b.m), 0.f, 0.f};
  if (a.s != 0.f) {
    const float d = shift(a.m, r.m, c), f = ex2_approx(d);
    r.s = f * a.s;
    r.u = f == 0.f ? 0.f : f * (a.u + d * a.s);
  }
  if (b.s != 0.f) {
    const float d = shift(b.m, r.m, c), f = ex2_approx(d);
    r.s += f * b.s;
    r.u += f == 0.f ? 0.f : f * (b.u + d * b.s);
  }
  return r;
}

__device__ __forceinline__ void add_value(Stats& st, float x, float c) {
  Stats one = {x, 0.f, 0.f};
  if (x != -INFINITY) {
    const float y = exponent(x, x, c);       // what fp32(c x) leaves out; NaN for +inf
    one.s = ex2_approx(y);
    one.u = one.s * y;
  }
  st = join(st, one, c);
}

// The larger, or smaller, of two values, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest of a group of vectors, NaN where one is.
template <typename T, int N>
__device__ __forceinline__ float group_max(const uint4 (&r)[N]) {
  if constexpr (sizeof(T) == 2) {
    auto h = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
    __nv_bfloat162 v;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const __nv_bfloat162 p = __hmax2_nan(__hmax2_nan(h(r[i].x), h(r[i].y)), __hmax2_nan(h(r[i].z), h(r[i].w)));
      v = i ? __hmax2_nan(v, p) : p;
    }
    return max_nan(__low2float(v), __high2float(v));
  } else {
    float v = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
      v = max_nan(v, max_nan(max_nan(__uint_as_float(r[i].x), __uint_as_float(r[i].y)),
                             max_nan(__uint_as_float(r[i].z), __uint_as_float(r[i].w))));
    return v;
  }
}

// A thread's statistics while it walks: s and u in two halves each.
struct Sums {
  float s0, s1, u0, u1;

  // kCareful: some of the values are -inf or so low that y is not finite, or c m is far.
  template <bool kCareful>
  __device__ __forceinline__ void add(float x0, float x1, float m, float cm, float c, bool far) {
    float y0 = fmaf(x0, c, -cm), y1 = fmaf(x1, c, -cm);
    if constexpr (kCareful) {
      y0 = fmaxf(far ? (x0 - m) * c : y0, kLeast);
      y1 = fmaxf(far ? (x1 - m) * c : y1, kLeast);
    }
    const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
    s0 += e0;
    s1 += e1;
    u0 = fmaf(e0, y0, u0);
    u1 = fmaf(e1, y1, u1);
  }
  template <typename T, bool kCareful, int N>
  __device__ __forceinline__ void add_group(const uint4 (&r)[N], float m, float cm, float c) {
    const bool far = kCareful && is_far(cm);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) add<kCareful>(bf16_lo(w[j]), bf16_hi(w[j]), m, cm, c, far);
      } else {
        add<kCareful>(__uint_as_float(w[0]), __uint_as_float(w[1]), m, cm, c, far);
        add<kCareful>(__uint_as_float(w[2]), __uint_as_float(w[3]), m, cm, c, far);
      }
    }
  }
};

// kAgain: the careful path reads a group's vectors once more, one at a time, which keeps
// the code short (it fits the instruction cache); else it takes them from registers.
template <bool kAgain>
struct Walk {
  bool low = false;                  // a group with values for the careful path has come, or c m is far
  float best = -INFINITY;            // the largest value
  float m = -INFINITY, cm = NAN;     // reference of the sums; NaN: no value yet, or far
  Sums sum = {0.f, 0.f, 0.f, 0.f};

  // Returns the group's largest value.  again(i): the group's i-th vector once more.
  template <typename T, int N, typename F>
  __device__ __forceinline__ float add(const uint4 (&r)[N], float c, F again) {
    const float most = group_max<T>(r);
    best = max_nan(best, most);
    if (!(fmaf(most, c, -cm) <= 4.f)) {
      if (most == -INFINITY) return most;              // adds nothing
      const float to = max_nan(m, most);
      if (m != -INFINITY) {
        const float d = fmaxf(shift(m, to, c), kLeast), f = ex2_approx(d);
        sum.u0 = f * fmaf(d, sum.s0, sum.u0);
        sum.u1 = f * fmaf(d, sum.s1, sum.u1);
        sum.s0 *= f;
        sum.s1 *= f;
      }
      m = to;
      low = low && cm == cm;         // far from here no longer
      cm = __fmul_rn(m, c);
      if (is_far(cm)) {
        cm = NAN;
        low = true;
      }
      if (!(to < INFINITY)) sum.s0 = NAN;
    }
    if (!low) {
      const Sums before = sum;
      sum.add_group<T, false>(r, m, cm, c);
      if (fabsf(sum.u0 + sum.u1) < INFINITY) return most;
      low = true;                    // 0 * -inf: again, with care
      sum = before;
    }
    if constexpr (kAgain) {
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        const uint4 v[1] = {again(i)};
        sum.add_group<T, true>(v, m, cm, c);
      }
    } else {
      sum.add_group<T, true>(r, m, cm, c);
    }
    return most;
  }

  // The same of a group of which only the first n vectors may be there (all: they are).
  template <typename T, int N, typename F>
  __device__ __forceinline__ float add_some(const uint4 (&r)[N], bool all, float c, F again, int n) {
    if (all || (c > kFillerLeast && c < kFillerScale && group_max<T>(r) > kFillerMost)) return add<T>(r, c, again);
    float most = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < N && i < n; ++i) {
      const uint4 one[1] = {again(i)};
      most = max_nan(most, add<T>(one, c, [&](int) { return again(i); }));
    }
    return most;
  }

  __device__ __forceinline__ Stats stats() const { return {m, sum.s0 + sum.s1, sum.u0 + sum.u1}; }
};

// ------------------------------------------------------------ the k largest

// What a walk leaves of a row, NT threads at most: order bits of each thread's maximum
// (0: it had no vector) and the maxima of its pieces.
template <int NT>
struct Maxima {
  uint32_t best[NT];
  float piece[kPieces][NT];
};
// What the selecting warp works in.
struct Scratch {
  unsigned long long cand[kCand];
  uint16_t hit[kMaxTop + kTieThreads];             // threads that reach t
  uint16_t read[kMaxTop * kPieces + kTiePieces];   // pieces to be read again: above t, then t
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

// A t that k of up to 32 kPer values reach: the k-th largest of them, or one that exactly
// k reach.  bits(i): the order bits of this lane's i-th value, 0 for none.  0: fewer than k
// values.  The bits below kLow are the same in every value of the type and its sign.
template <typename T, int kPer, typename F>
__device__ __forceinline__ uint32_t kth_largest(F bits, int k) {
  constexpr int kLow = sizeof(T) == 2 ? 16 : 0;
  uint32_t key[kPer], most = 0, least = 0xffffffffu;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    key[i] = bits(i);
    most = max(most, key[i]);
    if (key[i]) {
      least = min(least, key[i]);
      ++n;
    }
  }
  if (__reduce_add_sync(0xffffffffu, n) < k) return 0;
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  if (most == least) return most;
  // the bits that all share, then one after the other
  int bit = 31 - __clz(most ^ least);
  uint32_t t = most & (0xfffffffeu << bit);
#pragma unroll 1
  for (; bit >= kLow; --bit) {
    const uint32_t c = t | (1u << bit);
    n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) n += key[i] >= c;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= k) t = c;
    if (n == k) return t;
  }
  // a negative value's low bits are ones, NaN's too
  if (kLow && t >= 0xffff0000u) return 0xffffffffu;
  if (kLow && !(t & 0x80000000u)) t |= (1u << kLow) - 1;
  return t;
}

// The k largest of the slice in order, to `out` (0 where it has fewer), by one warp.
// The walk was that of nt threads (a power of two) in `groups` groups of kGroup vectors,
// `span` groups to a piece.  kMany: k may be close to nt, with many values above t.
template <typename T, int NT, int kGroup, bool kMany>
__device__ void k_largest(const Slice<T>& sl, const Maxima<NT>& mx, int nt, int groups, int span, int k, Scratch& sc,
                          unsigned long long* out) {
  constexpr int VEC = kVec16<T>;
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1;
  const uint32_t t = kth_largest<T, NT / 32>([&](int i) { return i * 32 < nt ? mx.best[i * 32 + lane] : 0u; }, k);
  const int pieces = (groups + span - 1) / span;

  // the threads above t (at most k) and, if they are few, those at t; then their pieces.
  // Many at t (a row of equal values, or of -inf): ties are looked for in the order of
  // the columns instead.
  int above = 0, equal = 0, hits = 0, at_t = 0;
  for (int b = 0; b < nt && t; b += 32) at_t += __popc(__ballot_sync(kAll, mx.best[b + lane] == t));
  const bool few = at_t <= kTieThreads;
  for (int b = 0; b < nt && t; b += 32) {
    const uint32_t best = mx.best[b + lane];
    const bool hit = best > t || (few && best == t);
    const unsigned who = __ballot_sync(kAll, hit);
    if (hit) sc.hit[hits + __popc(who & below)] = static_cast<uint16_t>(b + lane);
    hits += __popc(who);
  }
  __syncwarp();
  const float per = 1.f / pieces;            // at most 2^10 of them: exact after the floor
  for (int u0 = 0; u0 < hits * pieces; u0 += 32) {
    const int u = u0 + lane, i = static_cast<int>((u + 0.5f) * per), p = u - i * pieces;
    const int who = u < hits * pieces ? sc.hit[i] : 0;
    const bool in = u < hits * pieces && sl.v0 + p * span * kGroup * nt + who < sl.v1;
    const uint32_t bits = in ? order_bits(mx.piece[p][who]) : 0u;
    const unsigned up = __ballot_sync(kAll, bits > t), eq = __ballot_sync(kAll, bits == t);
    const uint16_t id = static_cast<uint16_t>(p * nt + who);
    if (bits > t) sc.read[above + __popc(up & below)] = id;
    above += __popc(up);
    const int at = equal + __popc(eq & below);
    if (bits == t && at < kTiePieces) sc.read[kMaxTop * kPieces + at] = id;
    equal += __popc(eq);
  }
  __syncwarp();
  const bool take_ties = t && few && equal <= kTiePieces;
  const int todo = above + (take_ties ? equal : 0);

  // values above `floor` wait in sc.cand; where it fills up, the k largest of them stay
  int n = 0;
  unsigned long long floor = static_cast<unsigned long long>(t) << 32 | (t && !take_ties ? 0xffffffffu : 0u);
  auto order = [&] {
    __syncwarp();
    // Each is compared with all: n^2 / 32 steps.  Many are cut down to those that reach
    // the k-th value first: [4096][1000] fp32 with 64 alternatives 83 us, 291 without.
    // (Where k is far below nt it is not worth its code: [4096][32003] 132 us, 141 with.)
    if (kMany && n > kOrderAtOnce) {
      const uint32_t kth = kth_largest<T, kCand / 32>(
          [&](int i) { return i * 32 + lane < n ? static_cast<uint32_t>(sc.cand[i * 32 + lane] >> 32) : 0u; }, k);
      int kept = 0;
      for (int i = 0; i < n; i += 32) {
        const unsigned long long key = i + lane < n ? sc.cand[i + lane] : 0ull;
        const bool keep = i + lane < n && static_cast<uint32_t>(key >> 32) >= kth;
        const unsigned who = __ballot_sync(kAll, keep);
        __syncwarp();                              // read before the place is written
        if (keep) sc.cand[kept + __popc(who & below)] = key;
        kept += __popc(who);
      }
      n = kept;
      __syncwarp();
    }
    for (int i = lane; i < n; i += 32) {
      const unsigned long long key = sc.cand[i];
      int place = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) place += sc.cand[j] > key;
      if (place < k) out[place] = key;
    }
    __syncwarp();
  };
  auto see = [&](bool in, uint32_t b, int col) {
    const unsigned long long key = order_key(b, col);
    const unsigned who = __ballot_sync(kAll, in && key > floor);
    if (who >> lane & 1u) sc.cand[n + __popc(who & below)] = key;
    n += __popc(who);
  };
  // a vector a lane: first which of its values reach t at all (NaN does), then those,
  // one a lane at a time
  const float least = t ? from_order_bits(t) : -INFINITY;
  auto see_vector = [&](bool in, const uint4& r, int v) {
    float f[VEC];
    Raw<T, VEC> raw;
    raw.v = r;
    widen<T, VEC>(raw, f);
    unsigned hits = 0;
#pragma unroll
    for (int j = 0; j < VEC; ++j) hits |= !(f[j] < least) ? 1u << j : 0u;
    if (!in) hits = 0;
    const int col = sl.column(v);
    while (__any_sync(kAll, hits)) {
      const int j = __ffs(hits) - 1;
      float x = f[0];
#pragma unroll
      for (int i = 1; i < VEC; ++i) x = i == j ? f[i] : x;
      see(hits, order_bits(x), col + j);
      hits &= hits - 1;
    }
    if (n > kCand - 32 * VEC) {
      order();
      n = n < k ? n : k;
      for (int i = lane; i < n; i += 32) sc.cand[i] = out[i];
      if (n == k) floor = out[k - 1];
      __syncwarp();
    }
  };
  // vectors of the pieces, or, t = 0, all of them: four a lane on their way
  const int each = span * kGroup, units = t ? todo * each : sl.v1 - sl.v0, log_nt = 31 - __clz(nt);
  for (int u0 = 0; u0 < units; u0 += 4 * 32) {
    uint4 r[4];
    int v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int u = u0 + q * 32 + lane;
      v[q] = sl.v1;
      if (u < units) {
        if (t) {
          const int i = static_cast<int>(static_cast<unsigned>(u) / static_cast<unsigned>(each));
          const int id = sc.read[i < above ? i : kMaxTop * kPieces + i - above], p = id >> log_nt;
          v[q] = sl.v0 + ((p * each + u - i * each) << log_nt) + (id & (nt - 1));
        } else {
          v[q] = sl.v0 + u;
        }
      }
      r[q] = v[q] < sl.v1 ? load_block(sl.row, sl.column(v[q])) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (u0 + q * 32 >= units) break;
      see_vector(v[q] < sl.v1, r[q], v[q]);
    }
  }
  {
    const bool in = lane < sl.loose();
    const int col = in ? sl.loose_column(lane) : 0;
    see(in, in ? order_bits(to_f32(sl.row[col])) : 0u, col);
  }
  if (t && !take_ties && n < k) {
    // values equal to t by column: head, vectors, tail
    const int need = k - n, steps = (sl.v1 - sl.v0 + 31) / 32;
    int have = 0;
    for (int i = -1; i <= steps && have < need; ++i) {
      uint32_t b[VEC] = {};
      int col = 0, count = 0;
      if (i < 0 || i == steps) {
        const int in = i < 0 ? (sl.first ? sl.head : 0) : (sl.last ? sl.tail : 0);
        if (lane < in) {
          col = i < 0 ? lane : sl.head + sl.nvec * VEC + lane;
          b[0] = order_bits(to_f32(sl.row[col]));
        }
      } else if (sl.v0 + i * 32 + lane < sl.v1) {
        col = sl.column(sl.v0 + i * 32 + lane);
        block_bits<T>(load_block(sl.row, col), b);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) count += b[j] == t;
      int upto = count;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += o;
      }
      int at = have + upto - count;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (b[j] == t) {
          if (at < need) sc.cand[n + at] = order_key(t, col + j);
          ++at;
        }
      have += __shfl_sync(kAll, upto, 31);
    }
    n = have < need ? n + have : k;
  }
  order();
  for (int i = n + lane; i < k; i += 32) out[i] = 0;
  __syncwarp();
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

__device__ __forceinline__ void write_zeros(const ScoreFwdArgs& a, long long row, int tid, int nt) {
  for (int j = tid; j < a.M; j += nt) a.logprob[row * a.M + j] = 0.f;
  for (int j = tid; j < a.k; j += nt) {
    a.top[row * a.k + j] = 0.f;
    a.ids[row * a.k + j] = -1;
  }
  if (tid == 0) a.entropy[row] = a.lse[row] = 0.f;
}

// Groups to a piece.
__device__ __forceinline__ int span_of(int groups) { return (groups + kPieces - 1) / kPieces; }
// A thread's maxima of its pieces while it walks.
struct Pieces {
  float* at;            // of the current piece
  int span, left;       // groups to a piece, and of the current one
  float most = -INFINITY;
  template <int NT>
  __device__ __forceinline__ Pieces(Maxima<NT>& mx, int span_) : at(&mx.piece[0][threadIdx.x]), span(span_), left(span_) {}
  template <int NT>
  __device__ __forceinline__ void add(float x) {
    most = max_nan(most, x);
    *at = most;
    if (--left == 0) {
      left = span;
      at += NT;
      most = -INFINITY;
    }
  }
};

// The log probability of a value; ls = log2 s.  Where p is 1 to the last digits, ls may be
// a rounding below y.
__device__ __forceinline__ float log_prob(float x, const Stats& st, float ls, const ScoreFwdArgs& a) {
  const float y = exponent(x, st.m, a.c);
  const float lp = isinf(y) ? fmaf(x, a.scale, -(st.m * a.scale)) - kLn2 * ls   // y may leave fp32 where z does not
                            : kLn2 * (y - ls);
  return lp > 0.f ? 0.f : lp;
}

// A row's outputs from its statistics and its k largest, by one warp.
template <typename T>
__device__ __forceinline__ void write_row(const ScoreFwdArgs& a, long long row, const T* x, const Stats& st,
                                          const unsigned long long* sorted) {
  const int tid = threadIdx.x & 31, nt = 32;
  const float ls = st.s > 0.f ? log2f(st.s) : NAN;     // no finite value: NaN
  for (int j = tid; j < a.k; j += nt) {
    const unsigned long long key = sorted[j];
    a.top[row * a.k + j] = log_prob(from_order_bits(static_cast<uint32_t>(key >> 32)), st, ls, a);
    a.ids[row * a.k + j] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
  }
  for (int j = tid; j < a.M; j += nt) {
    const int t = a.tokens[row * a.M + j];
    float lp = 0.f;
    if (t >= 0 && t < a.V) lp = log_prob(to_f32(x[t]), st, ls, a);
    else if (t != -1 && a.status) report(a.status, kStInvalidArg, kWhereScore, static_cast<int>(row));
    a.logprob[row * a.M + j] = lp;
  }
  if (tid == 0) {
    const float cm = __fmul_rn(st.m, a.c);
    // z_m, and what the sums leave out of c m: lse, which the gradient starts from, is within
    // a step of its type however large it is
    const float rest = is_far(cm) ? 0.f : fmaf(st.m, a.c, -cm);
    a.lse[row] = fmaf(st.m, a.scale, kLn2 * (ls - rest));
    const float h = kLn2 * (ls - st.u / st.s);
    a.entropy[row] = h < 0.f ? 0.f : h;
  }
}

// The statistics of a warp's lanes together, in a fixed order: each is brought to the
// largest m once, then s and u add up.
__device__ __forceinline__ Stats warp_stats(Stats st, float c) {
  float m = st.m;
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (st.s != 0.f) {
    const float d = shift(st.m, m, c), f = ex2_approx(d);
    st.u = f == 0.f ? 0.f : f * fmaf(d, st.s, st.u);
    st.s *= f;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    st.s += __shfl_xor_sync(0xffffffffu, st.s, d);
    st.u += __shfl_xor_sync(0xffffffffu, st.u, d);
  }
  st.m = m;
  return st;
}
// The same of a CTA's warps, by one warp.
__device__ __forceinline__ Stats row_stats(const Stats* warps, int n, float c) {
  const int lane = threadIdx.x & 31;
  return warp_stats(lane < n ? warps[lane] : Stats{-INFINITY, 0.f, 0.f}, c);
}

// A row a cluster of a.split CTAs (1: no cluster).
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) score_fwd_kernel(const ScoreFwdArgs a) {
  __shared__ Maxima<kThreads> mx;
  __shared__ Scratch sc;
  __shared__ Stats warps[kThreads / 32];
  __shared__ Stats part[kMaxSplit];                         // of the row's CTAs, in CTA 0
  __shared__ unsigned long long list[kMaxSplit * kMaxTop];  // their k largest, in CTA 0
  constexpr int kGroup = 4;           // vectors a thread loads at a time
  const int split = a.split, rank = split > 1 ? blockIdx.x % split : 0;
  const long long row = blockIdx.x / split;
  const int nt = blockDim.x, tid = threadIdx.x;
  if (a.mask && !a.mask[row]) {
    if (rank == 0) write_zeros(a, row, tid, nt);
    return;
  }
  if (split > 1) cluster_arrive();         // CTA 0 is there before it is written to
  const T* x = static_cast<const T*>(a.x) + row * a.ld;
  const Slice<T> sl(x, a.V, rank, split);

  Walk<false> w;
  const int groups = (sl.v1 - sl.v0 + kGroup * nt - 1) / (kGroup * nt), span = span_of(groups);
  Pieces pieces(mx, span);
  for (int v = sl.v0 + tid; v < sl.v1; v += kGroup * nt) {
    auto again = [&](int i) { return v + i * nt < sl.v1 ? load_block(x, sl.column(v + i * nt)) : filler<T>(); };
    uint4 r[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) r[i] = again(i);
    const float most = w.add_some<T>(r, v + (kGroup - 1) * nt < sl.v1, a.c, again, (sl.v1 - v + nt - 1) / nt);
    pieces.add<kThreads>(most);
  }
  Stats st = w.stats();
  if (tid < sl.loose()) add_value(st, to_f32(x[sl.loose_column(tid)]), a.c);
  st = warp_stats(st, a.c);
  if ((tid & 31) == 0) warps[tid >> 5] = st;
  mx.best[tid] = sl.v0 + tid < sl.v1 ? order_bits(w.best) : 0u;
  __syncthreads();
  if (tid < 32) {
    st = row_stats(warps, nt / 32, a.c);
    if (a.k) k_largest<T, kThreads, kGroup, true>(sl, mx, nt, groups, span, a.k, sc, list);
  }
  __syncthreads();
  if (split > 1) {
    cluster_wait();
    if (rank) {
      for (int i = tid; i < a.k; i += nt) store_cta0(&list[rank * a.k + i], list[i]);
      if (tid == 0) {
        store_cta0(&part[rank].m, st.m);
        store_cta0(&part[rank].s, st.s);
        store_cta0(&part[rank].u, st.u);
      }
    }
    cluster_arrive();
    cluster_wait();
    if (rank) return;
    if (tid < 32) {
      const int lane = tid;
      st = warp_stats(lane == 0 ? st : lane < split ? part[lane] : Stats{-INFINITY, 0.f, 0.f}, a.c);
    }
    // a value's place: its own in its list and how many of each other list are larger
    for (int i = tid; i < split * a.k; i += nt) {
      const unsigned long long key = list[i];
      const int own = i / a.k;
      int place = i - own * a.k;
      for (int o = 0; o < split; ++o) {
        if (o == own) continue;
        int lo = 0, hi = a.k;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (list[o * a.k + mid] > key) lo = mid + 1;
          else hi = mid;
        }
        place += lo;
      }
      if (key && place < a.k) sc.cand[place] = key;
    }
    __syncthreads();
  }
  if (tid < 32) write_row(a, row, x, st, split > 1 ? sc.cand : list);
}

// ------------------------------------------------------------ many long rows
//
// Two CTAs an SM take rows in turn.  Eight warps walk: a thread's next vectors come by
// cp.async into its own places of a ring in shared memory, on into the CTA's next row.
// Three other warps, each for every third row, find the k largest and write a row's
// outputs while the walk goes on.  [16384][128256] bf16 behind a 62 % mask: 399 us, 97 %
// of the copy rate; 674 with a CTA a row that does one after the other.

constexpr int kRowThreads = 256;                  // that walk
constexpr int kSelect = 3;                        // warps that find the k largest
constexpr int kRowAll = kRowThreads + 32 * kSelect;
constexpr int kRowCtas = 2;       // an SM
// Groups of vectors on their way: kGroup vectors are walked at a time.  Eight at a time
// take 10 % fewer instructions a value than four (4096 rows of 128256 bf16 with eight
// alternatives 176 us and 184), but need rows of more than two groups of 2048 vectors.
template <int kGroup>
constexpr int kRingGroups = kGroup == 8 ? 2 : 3;
template <int kGroup>
constexpr int kRingBytes = kRingGroups<kGroup> * kGroup * kRowThreads * 16;

// Barriers of the walking warps and a selecting one: `arrive` does not wait.
__device__ __forceinline__ void barrier_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kRowThreads + 32) : "memory");
}
__device__ __forceinline__ void barrier_arrive(int id) {
  __threadfence_block();
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kRowThreads + 32) : "memory");
}

__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The first active row of r, r + step, ... (N or more: none).
__device__ __forceinline__ long long active_row(const ScoreFwdArgs& a, long long r, long long step) {
  if (!a.mask) return r;
  const int lane = threadIdx.x & 31;
  while (r < a.N) {
    const long long mine = r + lane * step;
    const unsigned on = __ballot_sync(0xffffffffu, mine < a.N && a.mask[mine]);
    if (on) return r + (__ffs(on) - 1) * step;
    r += 32 * step;
  }
  return r;
}

struct RowShared {
  Maxima<kRowThreads> mx[kSelect];                 // of kSelect rows in turn
  Stats warps[kSelect][kRowThreads / 32];
  Scratch scratch[kSelect];
  unsigned long long list[kSelect][kMaxTop];
};
template <int kGroup>
constexpr int kRowBytes = kRingBytes<kGroup> + static_cast<int>(sizeof(RowShared));

template <typename T, int kGroup>
__global__ void __launch_bounds__(kRowAll, kRowCtas) score_rows_kernel(const ScoreFwdArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* ring = reinterpret_cast<uint4*>(smem);    // [kAhead][kGroup][kRowThreads]
  RowShared& sh = *reinterpret_cast<RowShared*>(smem + kRingBytes<kGroup>);
  constexpr int VEC = kVec16<T>, kStep = kGroup * kRowThreads, kAhead = kRingGroups<kGroup>;
  constexpr int kFull = 1, kEmpty = 1 + kSelect;   // barriers: + turn
  const int tid = threadIdx.x;
  const long long step = gridDim.x;
  const T* base = static_cast<const T*>(a.x);
  if (a.mask)
    for (long long r = blockIdx.x + tid * step; r < a.N; r += kRowAll * step)
      if (!a.mask[r]) write_zeros(a, r, 0, 1);

  long long row = active_row(a, blockIdx.x, step);
  int turn = 0;
  if (tid >= kRowThreads) {
    // every kSelect-th row of the CTA's
    turn = (tid - kRowThreads) >> 5;
    auto on = [&](long long r, int n) {
      for (int i = 0; i < n && r < a.N; ++i) r = active_row(a, r + step, step);
      return r;
    };
    row = on(row, turn);
    Scratch& sc = sh.scratch[turn];
    unsigned long long* list = sh.list[turn];
    while (row < a.N) {
      const long long next = on(row, kSelect);
      const Slice<T> sl(base + row * a.ld, a.V, 0, 1);
      const int groups = (sl.nvec + kStep - 1) / kStep;
      barrier_sync(kFull + turn);
      if (a.k) k_largest<T, kRowThreads, kGroup, false>(sl, sh.mx[turn], kRowThreads, groups, span_of(groups), a.k, sc, list);
      const Stats st = row_stats(sh.warps[turn], kRowThreads / 32, a.c);
      __syncwarp();
      if (next < a.N) barrier_arrive(kEmpty + turn);
      write_row(a, row, sl.row, st, list);
      __syncwarp();
      row = next;
    }
    return;
  }
  if (row >= a.N) return;
  // copies to a slot the group of vectors from `from` on, `left` of them this thread's
  auto issue = [&](int to, const T* from, int left) {
    uint4* p = ring + to * kStep + tid;
    if (left > (kGroup - 1) * kRowThreads) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) copy_async(p + k * kRowThreads, from + k * kRowThreads * VEC);
    } else {
#pragma unroll 1
      for (int k = 0; k * kRowThreads < left; ++k) copy_async(p + k * kRowThreads, from + k * kRowThreads * VEC);
    }
    copies_commit();
  };
  Slice<T> sl(base + row * a.ld, a.V, 0, 1);
#pragma unroll 1
  for (int g = 0; g < kAhead; ++g)
    issue(g, sl.row + sl.head + (tid + g * kStep) * VEC, sl.nvec - tid - g * kStep);

  int slot = 0, done = 0;
#pragma unroll 1
  while (true) {
    const long long next = active_row(a, row + step, step);
    const Slice<T> after(base + (next < a.N ? next : row) * a.ld, a.V, 0, 1);
    const int groups = (sl.nvec + kStep - 1) / kStep, span = span_of(groups);
    // kAhead groups from here: of this row, then of the next one (rows have as many
    // groups or one more or less; more than kAhead)
    const T* from = sl.row + sl.head + (tid + kAhead * kStep) * VEC;
    int here = sl.nvec - tid;          // this thread's vectors: every kRowThreads-th of them
    int ahead = here - kAhead * kStep;
    if (done >= kSelect) barrier_sync(kEmpty + turn);
    Walk<true> w;
    Pieces pieces(sh.mx[turn], span);
#pragma unroll 1
    for (int g = groups; g > 0; --g) {
      copies_wait<kAhead - 1>();
      const uint4* in = ring + slot * kStep + tid;
      const bool all = here > (kGroup - 1) * kRowThreads;
      auto again = [&](int i) { return i * kRowThreads < here ? in[i * kRowThreads] : filler<T>(); };
      uint4 r[kGroup];
      if (all) {
#pragma unroll
        for (int k = 0; k < kGroup; ++k) r[k] = in[k * kRowThreads];
      } else {
#pragma unroll
        for (int k = 0; k < kGroup; ++k) r[k] = again(k);
      }
      const float most = w.add_some<T>(r, all, a.c, again, (here + kRowThreads - 1) / kRowThreads);
      pieces.add<kRowThreads>(most);
      if (g == kAhead) {
        from = after.row + after.head + tid * VEC;
        ahead = (next < a.N ? after.nvec : 0) - tid;
      }
      issue(slot, from, ahead);
      from += kStep * VEC;
      ahead -= kStep;
      here -= kStep;
      slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
    Stats st = w.stats();
    if (tid < sl.loose()) add_value(st, to_f32(sl.row[sl.loose_column(tid)]), a.c);
    st = warp_stats(st, a.c);
    if ((tid & 31) == 0) sh.warps[turn][tid >> 5] = st;
    sh.mx[turn].best[tid] = tid < sl.nvec ? order_bits(w.best) : 0u;
    __syncwarp();
    barrier_arrive(kFull + turn);
    turn = turn + 1 == kSelect ? 0 : turn + 1;
    ++done;
    if (next >= a.N) break;
    row = next;
    sl = after;
  }
  copies_wait<0>();
}

// ----------------------------------------------------------------- backward

// Bound by its bytes: one read (of active rows) and one write, a few vectors a thread on
// their way.  [16384][128256] bf16 behind a 62 % mask 999 us, the copy rate.
// Where logits and their gradient lie differently to 16 bytes the stores are single elements:
// [4096][32003] bf16 out of rows of 32064 to dense ones 306 us, 91 between rows of one pitch
// (fp32 162 and 159).
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
    const float d = max_nan(min_nan(fmaf(xv, a.scale, -lse), 0.f), kLeast);
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

template <typename T, int kGroup>
cudaError_t launch_rows(const ScoreFwdArgs& a, int num_sms, cudaStream_t s) {
  const cudaError_t e = allow_smem<score_rows_kernel<T, kGroup>>(kRowBytes<kGroup>);
  if (e != cudaSuccess) return e;
  score_rows_kernel<T, kGroup><<<kRowCtas * num_sms, kRowAll, kRowBytes<kGroup>, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_score_fwd(const ScoreFwdArgs& args, int is_bf16, int num_sms, cudaStream_t s) {
  if (args.N == 0) return cudaSuccess;
  ScoreFwdArgs a = args;
  const long long nvec = a.V / (is_bf16 ? 8 : 4);
  if (a.N > kRowCtas * static_cast<long long>(num_sms) && nvec > 3 * 4 * kRowThreads + 8) {
    return nvec > 2 * 8 * kRowThreads + 8   // more groups than are on their way, wherever a row starts
               ? is_bf16 ? launch_rows<__nv_bfloat16, 8>(a, num_sms, s) : launch_rows<float, 8>(a, num_sms, s)
               : is_bf16 ? launch_rows<__nv_bfloat16, 4>(a, num_sms, s) : launch_rows<float, 4>(a, num_sms, s);
  }
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
