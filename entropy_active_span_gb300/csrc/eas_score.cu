// Scores of logits that exist: log probabilities of given tokens, entropy, the top
// alternatives of each row, and the gradient of all of them at the logits.
//
// With c = scale log2 e, a row's statistics are kept in base 2:
//   y = c x - fp32(c m),  s = sum 2^y,  u = sum 2^y y,
//   lse = ln2 (fp32(c m) + log2 s),  logp(t) = ln2 (y_t - log2 s),
//   H = ln2 (log2 s - u / s),
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
// Backward, with G = sum of a row's g_j and p = 2^(c x - log2 e lse):
//   dx_v = scale (sum_j g_j [v == t_j] - p_v (G + g_H (z_v - lse + H))).
#include "eas_device.cuh"
#include "eas_launch.cuh"
#include "eas_ops.h"
#include "eas_vec.cuh"

namespace eas {

namespace {

constexpr int kThreads = 512;     // at most
constexpr int kGroup = 4;         // vectors a thread loads at a time
constexpr int kCand = 512;        // values above t that are kept
constexpr int kTies = 128;        // and values equal to it
constexpr int kPieces = 8;        // of a thread's part
constexpr int kTiePieces = 512;   // pieces whose maximum is t that are read again
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

// c x - fp32(c m); where c m leaves fp32, c (x - m).
__device__ __forceinline__ float exponent(float x, float m, float c) {
  const float cm = __fmul_rn(m, c);
  return fabsf(cm) < INFINITY ? fmaf(x, c, -cm) : (x - m) * c;
}
// What to add to an exponent below m to have one below n >= m.
__device__ __forceinline__ float shift(float m, float n, float c) {
  const float d = __fmul_rn(m, c) - __fmul_rn(n, c);
  return d <= 0.f ? d : (m - n) * c;
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

  // kCareful: some of the values are -inf or so low that y is not finite.
  template <bool kCareful>
  __device__ __forceinline__ void add(float x0, float x1, float m, float cm, float c) {
    const float y0 = kCareful ? fmaxf(exponent(x0, m, c), kLeast) : fmaf(x0, c, -cm);
    const float y1 = kCareful ? fmaxf(exponent(x1, m, c), kLeast) : fmaf(x1, c, -cm);
    const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
    s0 += e0;
    s1 += e1;
    u0 = fmaf(e0, y0, u0);
    u1 = fmaf(e1, y1, u1);
  }
  template <typename T, bool kCareful, int N>
  __device__ __forceinline__ void add_group(const uint4 (&r)[N], float m, float cm, float c) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) add<kCareful>(bf16_lo(w[j]), bf16_hi(w[j]), m, cm, c);
      } else {
        add<kCareful>(__uint_as_float(w[0]), __uint_as_float(w[1]), m, cm, c);
        add<kCareful>(__uint_as_float(w[2]), __uint_as_float(w[3]), m, cm, c);
      }
    }
  }
};

struct Walk {
  float best = -INFINITY;            // the largest value
  float m = -INFINITY, cm = 0.f;     // reference of the sums
  Sums sum = {0.f, 0.f, 0.f, 0.f};

  // Returns the group's largest value.
  template <typename T, int N>
  __device__ __forceinline__ float add(const uint4 (&r)[N], float c) {
    const float most = group_max<T>(r);
    best = max_nan(best, most);
    if (!(fmaf(most, c, -cm) <= 4.f) || m == -INFINITY) {
      if (most == -INFINITY) return most;              // nothing but -inf so far
      const float to = max_nan(m, most);
      if (m != -INFINITY) {
        const float d = fmaxf(shift(m, to, c), kLeast), f = ex2_approx(d);
        sum.u0 = f * fmaf(d, sum.s0, sum.u0);
        sum.u1 = f * fmaf(d, sum.s1, sum.u1);
        sum.s0 *= f;
        sum.s1 *= f;
      }
      m = to;
      cm = __fmul_rn(m, c);
      if (!(to < INFINITY)) sum.s0 = NAN;
    }
    const Sums before = sum;
    sum.add_group<T, false>(r, m, cm, c);
    if (!(fabsf(sum.u0 + sum.u1) < INFINITY)) {        // 0 * -inf: again, with care
      sum = before;
      sum.add_group<T, true>(r, m, cm, c);
    }
    return most;
  }

  __device__ __forceinline__ Stats stats() const { return {m, sum.s0 + sum.s1, sum.u0 + sum.u1}; }
};

// ------------------------------------------------------------ the k largest

// NT: threads of the CTA, at most.
template <int NT>
struct Shared {
  uint32_t best[NT];                              // order bits of the threads' maxima
  unsigned long long cand[kCand];
  unsigned long long tie[kTies];
  float piece[kPieces][NT];                       // maxima of the threads' pieces
  uint16_t read[kMaxTop * kPieces + kTiePieces];  // pieces to be read again: above t, then t
  int scan[NT / 32];
  uint32_t t;
  int n_above, n_tie, n_pieces, n_tie_pieces;
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
template <typename T, int kWarps>
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
template <typename T, int NT>
__device__ void first_ties(const Slice<T>& sl, Shared<NT>& sm, uint32_t t, int from, int need) {
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

// The k largest of the slice in order, to `out` (0 where it has fewer).  `best`: the
// thread's maximum over its vectors (if it has any), in `groups` groups, `span` to a
// piece.
template <typename T, int NT>
__device__ void k_largest(const Slice<T>& sl, Shared<NT>& sm, float best, int groups, int span, int k,
                          unsigned long long* out) {
  constexpr int VEC = kVec16<T>;
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t mine = sl.v0 + tid < sl.v1 ? order_bits(best) : 0u;
  sm.best[tid] = mine;
  if (tid == 0) sm.n_above = sm.n_tie = sm.n_pieces = sm.n_tie_pieces = 0;
  __syncthreads();
  if (warp == 0) {
    const uint32_t t = kth_of_maxima<T, NT / 32>(sm.best, nt, k, lane);
    if (lane == 0) sm.t = t;
  }
  __syncthreads();
  uint32_t t = sm.t;
  // fewer than k threads have pieces above t
  if (mine >= t && mine) {
    const int pieces = (groups + span - 1) / span;
    for (int p = 0; p < pieces; ++p) {
      if (sl.v0 + p * span * kGroup * nt + tid >= sl.v1) break;
      const uint32_t b = order_bits(sm.piece[p][tid]);
      const uint16_t id = static_cast<uint16_t>(p * nt + tid);
      if (b > t && t) {
        sm.read[atomicAdd(&sm.n_pieces, 1)] = id;
      } else if (b == t) {
        const int at = atomicAdd(&sm.n_tie_pieces, 1);
        if (at < kTiePieces) sm.read[kMaxTop * kPieces + at] = id;
      }
    }
  }
  __syncthreads();
  // many pieces with the same maximum (a row of equal values, or of -inf): the ties are
  // looked for in the order of the columns instead.  t = 0: every value is above it.
  const int above = t ? sm.n_pieces : 0, equal = sm.n_tie_pieces;
  const bool take_ties = t && equal <= kTiePieces;
  const int pieces = above + (take_ties ? equal : 0);
  auto see = [&](uint32_t b, int col) {
    if (b > t) push(sm.cand, &sm.n_above, kCand, b, col);
    else if (take_ties && b == t) push(sm.tie, &sm.n_tie, kTies, b, col);
  };
  // kGroup lanes a piece
  for (int i = tid / kGroup; i < pieces; i += nt / kGroup) {
    const int id = sm.read[i < above ? i : kMaxTop * kPieces + i - above], p = id / nt;
    for (int g = 0; g < span; ++g) {
      const int v = sl.v0 + ((p * span + g) * kGroup + tid % kGroup) * nt + id - p * nt;
      if (v >= sl.v1) break;
      uint32_t b[VEC];
      const int col = sl.column(v);
      block_bits<T>(load_block(sl.row, col), b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) see(b[j], col + j);
    }
  }
  if (t == 0) {
    for_all(sl, see);
  } else if (tid < sl.loose()) {
    const int col = sl.loose_column(tid);
    see(order_bits(to_f32(sl.row[col])), col);
  }
  __syncthreads();
  int n = sm.n_above;
  const int ties = sm.n_tie;
  bool look = t != 0 && n < k && !(take_ties && ties <= kTies);
  if (n > kCand) {
    // the few pieces that reach t hold too many values above it (a row whose large values
    // lie in few pieces): the k-th largest value itself, bit by bit
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

__device__ __forceinline__ void write_zeros(const ScoreFwdArgs& a, long long row, int tid, int nt) {
  for (int j = tid; j < a.M; j += nt) a.logprob[row * a.M + j] = 0.f;
  for (int j = tid; j < a.k; j += nt) {
    a.top[row * a.k + j] = 0.f;
    a.ids[row * a.k + j] = -1;
  }
  if (tid == 0) a.entropy[row] = a.lse[row] = 0.f;
}

// Groups to a piece, and the maximum of the thread's piece that group g belongs to.
__device__ __forceinline__ int span_of(int groups) { return (groups + kPieces - 1) / kPieces; }
template <int NT>
__device__ __forceinline__ void keep_piece(Shared<NT>& sm, int g, int span, float most) {
  float& p = sm.piece[g / span][threadIdx.x];
  p = g % span ? max_nan(p, most) : most;
}

// The log probability of a value; ls = log2 s.
__device__ __forceinline__ float log_prob(float x, const Stats& st, float ls, const ScoreFwdArgs& a) {
  const float y = exponent(x, st.m, a.c);
  return isinf(y) ? fmaf(x - st.m, a.scale, -kLn2 * ls) : kLn2 * (y - ls);   // c x may leave fp32 where scale x does not
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
    a.lse[row] = fabsf(cm) < INFINITY ? kLn2 * (cm + ls) : fmaf(kLn2, ls, st.m * a.scale);
    a.entropy[row] = kLn2 * (ls - st.u / st.s);
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
  __shared__ Shared<kThreads> sm;
  __shared__ Stats warps[kThreads / 32];
  __shared__ Stats part[kMaxSplit];                         // of the row's CTAs, in CTA 0
  __shared__ unsigned long long list[kMaxSplit * kMaxTop];  // their k largest, in CTA 0
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

  Walk w;
  const int groups = (sl.v1 - sl.v0 + kGroup * nt - 1) / (kGroup * nt), span = span_of(groups);
  int g = 0;
  for (int v = sl.v0 + tid; v < sl.v1; v += kGroup * nt, ++g) {
    uint4 r[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (v + i * nt < sl.v1) r[i] = load_block(x, sl.column(v + i * nt));
    float most;
    if (v + (kGroup - 1) * nt < sl.v1) {
      most = w.add<T>(r, a.c);
    } else {
      const uint4 one[1] = {r[0]};
      most = w.add<T>(one, a.c);
#pragma unroll
      for (int i = 1; i < kGroup - 1; ++i)
        if (v + i * nt < sl.v1) {
          const uint4 next[1] = {r[i]};
          most = max_nan(most, w.add<T>(next, a.c));
        }
    }
    if (a.k) keep_piece(sm, g, span, most);
  }
  Stats st = w.stats();
  if (tid < sl.loose()) add_value(st, to_f32(x[sl.loose_column(tid)]), a.c);
  st = warp_stats(st, a.c);
  if ((tid & 31) == 0) warps[tid >> 5] = st;
  if (a.k) k_largest(sl, sm, w.best, groups, span, a.k, list);
  __syncthreads();
  if (tid < 32) st = row_stats(warps, nt / 32, a.c);
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
      if (key && place < a.k) sm.cand[place] = key;
    }
    __syncthreads();
  }
  if (tid < 32) write_row(a, row, x, st, split > 1 ? sm.cand : list);
}

// ------------------------------------------------------------ many long rows
//
// Four CTAs an SM take rows in turn.  A thread's next vectors come by cp.async into its
// own places of a ring in shared memory, on into the CTA's next row while the k
// largest of this one are found: the loads never pause.  [16384][128256] bf16 behind
// a 62 % mask: 674 us with a CTA a row.

constexpr int kRowThreads = 256;
constexpr int kRowCtas = 4;       // an SM
constexpr int kRingGroups = 2;    // groups of vectors on their way
constexpr int kRingBytes = kRingGroups * kGroup * kRowThreads * 16;

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

template <typename T>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) score_rows_kernel(const ScoreFwdArgs a) {
  extern __shared__ uint4 ring[];     // [kRingGroups][kGroup][kRowThreads]
  __shared__ Shared<kRowThreads> sm;
  // of two rows in turn: warp 0 writes a row's outputs while the others are in the next
  __shared__ unsigned long long list[2][kMaxTop];
  __shared__ Stats warps[2][kRowThreads / 32];
  constexpr int VEC = kVec16<T>, kStep = kGroup * kRowThreads;
  const int tid = threadIdx.x;
  const long long step = gridDim.x;
  const T* base = static_cast<const T*>(a.x);
  if (a.mask)
    for (long long r = blockIdx.x + tid * step; r < a.N; r += kRowThreads * step)
      if (!a.mask[r]) write_zeros(a, r, 0, 1);

  // the next group to be copied: of row `coming`, `ahead` of its `whole` vectors done
  const long long first = active_row(a, blockIdx.x, step);
  long long coming = first;
  const T* body = nullptr;            // this thread's next vector
  int ahead = 0, whole = 0, slot_in = 0;
  auto open = [&] {
    if (coming >= a.N) return;
    const Slice<T> sl(base + coming * a.ld, a.V, 0, 1);
    body = sl.row + sl.head + tid * VEC;
    whole = sl.nvec;
    ahead = 0;
  };
  auto issue = [&] {
    if (coming < a.N) {
      uint4* to = ring + slot_in * kStep + tid;
      if (ahead + kStep <= whole) {
#pragma unroll
        for (int k = 0; k < kGroup; ++k) copy_async(to + k * kRowThreads, body + k * kRowThreads * VEC);
      } else {
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
          if (ahead + k * kRowThreads + tid < whole) copy_async(to + k * kRowThreads, body + k * kRowThreads * VEC);
      }
      body += kStep * VEC;
      ahead += kStep;
      if (ahead >= whole) {
        coming = active_row(a, coming + step, step);
        open();
      }
    }
    slot_in = slot_in + 1 == kRingGroups ? 0 : slot_in + 1;
    copies_commit();
  };
  open();
#pragma unroll 1
  for (int i = 0; i < kRingGroups; ++i) issue();

  long long row = first;
  int slot = 0, turn = 0;
#pragma unroll 1
  while (row < a.N) {
    const T* x = base + row * a.ld;
    const Slice<T> sl(x, a.V, 0, 1);
    Walk w;
    const int groups = (sl.nvec + kStep - 1) / kStep, span = span_of(groups);
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      copies_wait<kRingGroups - 1>();
      const uint4* from = ring + slot * kStep + tid;
      const int left = sl.nvec - g * kStep - tid;      // vectors of this thread: every kRowThreads-th of them
      float most = -INFINITY;
      if (left > (kGroup - 1) * kRowThreads) {
        uint4 r[kGroup];
#pragma unroll
        for (int k = 0; k < kGroup; ++k) r[k] = from[k * kRowThreads];
        most = w.add<T>(r, a.c);
      } else {
#pragma unroll 1
        for (int k = 0; k * kRowThreads < left; ++k) {
          const uint4 r[1] = {from[k * kRowThreads]};
          most = max_nan(most, w.add<T>(r, a.c));
        }
      }
      if (a.k) keep_piece(sm, g, span, most);
      issue();
      slot = slot + 1 == kRingGroups ? 0 : slot + 1;
    }
    Stats st = w.stats();
    if (tid < sl.loose()) add_value(st, to_f32(x[sl.loose_column(tid)]), a.c);
    st = warp_stats(st, a.c);
    if ((tid & 31) == 0) warps[turn][tid >> 5] = st;
    if (a.k) k_largest(sl, sm, w.best, groups, span, a.k, list[turn]);
    __syncthreads();
    if (tid < 32) write_row(a, row, x, row_stats(warps[turn], kRowThreads / 32, a.c), list[turn]);
    turn ^= 1;
    row = active_row(a, row + step, step);
  }
  copies_wait<0>();
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
  if (a.N > kRowCtas * static_cast<long long>(num_sms) && nvec >= 2 * kGroup * kRowThreads) {
    const auto kernel = is_bf16 ? score_rows_kernel<__nv_bfloat16> : score_rows_kernel<float>;
    const cudaError_t e = is_bf16 ? allow_smem<score_rows_kernel<__nv_bfloat16>>(kRingBytes)
                                  : allow_smem<score_rows_kernel<float>>(kRingBytes);
    if (e != cudaSuccess) return e;
    kernel<<<kRowCtas * num_sms, kRowThreads, kRingBytes, s>>>(a);
    return cudaGetLastError();
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
