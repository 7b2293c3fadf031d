// route.cu -- the router's choice from given logits, and its backward.
//
// Passage: dots.llm1 Technical Report, §Architecture "Mixture of Experts layer"
// and "Load balancing" (top-k of the affinities; the bias only decides the
// choice).  Sigmoid affinities, expert groups and a factor on the weights have no
// counterpart on the pages; the formulas stand in include/moe.h.
//
// A token takes a warp, lane l holding the EPL consecutive experts from l EPL on, or, where
// there are many of up to 128 experts, 8 or 16 lanes (few_lanes).
//
// The choice has to be the one of 64-bit arithmetic, at the price of 32 bits: scores are
// computed in FP32 with a bound on their error (margins below), and the order found stands
// where neighbouring scores differ by more than the bound, or by nothing in 64 bits
// either (equal logits and biases).  Where the check fails, about one token in a thousand,
// the few experts in question are ordered by their scores in 64 bits (refine), and so are
// groups (refine_groups); only tokens beyond FP32's range are done in 64 bits whole.
//
// What bounds the calls is a token's chain of steps and their issue: with 42 to 46 % of an SM's
// warps (registers) the forward takes 50 % of the issue slots up to 128 experts and 68 % with
// 256 in groups, the backward 40 to 45 %.  So a pick costs one reduction, a ballot and a few
// selects: each lane keeps its best four scores in order, and which expert a pick was is
// looked up once, by lane j for pick j.  Of 128 experts, 6 picks, FP32 logits, 8192 tokens
// took 7.0 us (1.2 TB/s) and 16384 11 (1.5 TB/s), their backward 7.1 us (2.5 TB/s); of 256
// experts in 8 groups, 8 picks, 16384 tokens 24 us and 11 us (3.1 TB/s).  Everything in 64
// bits, a warp a token, took 15, 26, 15, 80 and 33 us.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int RT_WARPS = 4;
constexpr int RT_EMAX = 256;  // experts
constexpr unsigned FULL = 0xffffffffu;

// Where FP32 gives way to 64 bits: below RT_TINY a pick's affinity is too near the subnormal
// numbers; below the sums, what was lost there counts in the weights or in probs.
constexpr float RT_TINY = 0x1p-100f;
constexpr float RT_SMALL_SUM = 0x1p-60f;  // of the picks' affinities
constexpr float RT_SMALL_ALL = 0x1p-20f;  // of all affinities

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  float* probs;
  int64_t T;
  int E, k, n_group, topk_group, group_top, renorm, softmax;
  int vec;  // rows of logits and probs can be read and written EPL experts at a time
  int few;  // a token takes a few lanes, not a warp
  float scale;
};

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

// FP32 values as unsigned numbers of the same order: -inf is 0x007fffff, zeros are equal.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}
constexpr uint32_t ORD_NEG_INF = 0x007fffffu;

// Largest of the warp's values, NaN left out (-inf where all are).
__device__ __forceinline__ float warp_max(float v) {
  return unordered(__reduce_max_sync(FULL, v != v ? ORD_NEG_INF : ordered(v)));
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// EPL neighbouring elements at once, as pieces of up to 16 bytes.
template <int BYTES>
struct Piece;
template <>
struct Piece<4> { using type = uint32_t; };
template <>
struct Piece<8> { using type = uint2; };
template <>
struct Piece<16> { using type = uint4; };

template <typename LT, int EPL>
struct __align__(16) Row {
  static constexpr int BYTES = EPL * sizeof(LT) < 16 ? EPL * sizeof(LT) : 16;
  static constexpr int N = EPL * sizeof(LT) / BYTES;
  using P = typename Piece<BYTES>::type;
  union {
    LT e[EPL];
    P p[N];
  };
  __device__ Row() {}
};

template <typename LT, int EPL>
__device__ __forceinline__ void load_row(float (&x)[EPL], const LT* row, int e0, int E, bool vec,
                                         float none) {
  if (vec && e0 < E) {
    Row<LT, EPL> r;
    const auto* p = reinterpret_cast<const typename Row<LT, EPL>::P*>(row + e0);
#pragma unroll
    for (int i = 0; i < r.N; ++i) r.p[i] = p[i];
#pragma unroll
    for (int q = 0; q < EPL; ++q) x[q] = load1(&r.e[q]);
  } else {
#pragma unroll
    for (int q = 0; q < EPL; ++q) x[q] = e0 + q < E ? load1(row + e0 + q) : none;
  }
}

template <typename LT, int EPL>
__device__ __forceinline__ void store_row(LT* row, const float (&x)[EPL], int e0, int E, bool vec) {
  if (vec) {
    if (e0 >= E) return;
    Row<LT, EPL> r;
#pragma unroll
    for (int q = 0; q < EPL; ++q) store1(&r.e[q], x[q]);
    auto* p = reinterpret_cast<typename Row<LT, EPL>::P*>(row + e0);
#pragma unroll
    for (int i = 0; i < r.N; ++i) p[i] = r.p[i];
  } else {
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if (e0 + q < E) store1(row + e0 + q, x[q]);
  }
}

// A lane's EPL values in a warp's shared memory: pieces of up to 16 bytes, the lanes' first
// ones before the second ones, so that the lanes' accesses do not meet in a bank.
template <int EPL>
__device__ __forceinline__ int slot(int lane, int q) {
  return EPL <= 4 ? lane * EPL + q : (q >> 2) * 128 + lane * 4 + (q & 3);
}
template <int EPL, typename V>
__device__ __forceinline__ void put(V* sh, int lane, const V (&v)[EPL]) {
  constexpr int N = EPL < 4 ? EPL : 4;
  using P = typename Piece<4 * N>::type;
#pragma unroll
  for (int i = 0; i < EPL / N; ++i) {
    union {
      P p;
      V e[N];
    } u;
#pragma unroll
    for (int j = 0; j < N; ++j) u.e[j] = v[i * N + j];
    *reinterpret_cast<P*>(sh + slot<EPL>(lane, i * N)) = u.p;
  }
}
template <int EPL, typename V>
__device__ __forceinline__ void get(const V* sh, int lane, V (&v)[EPL]) {
  constexpr int N = EPL < 4 ? EPL : 4;
  using P = typename Piece<4 * N>::type;
#pragma unroll
  for (int i = 0; i < EPL / N; ++i) {
    union {
      P p;
      V e[N];
    } u;
    u.p = *reinterpret_cast<const P*>(sh + slot<EPL>(lane, i * N));
#pragma unroll
    for (int j = 0; j < N; ++j) v[i * N + j] = u.e[j];
  }
}

// Shared memory of a warp.
union RouteShared {
  double f64[2 * RT_EMAX];  // scores and group scores
  struct {
    uint32_t key[RT_EMAX];  // ordered scores, by slot (refine: the experts in question)
    float p[RT_EMAX];       // affinities, by slot
    uint2 pick[32];         // key and lane of a pick
  } f32;
  struct {
    // of all the warp's tokens, by slot
    uint32_t key[2 * RT_EMAX];
    float p[2 * RT_EMAX];
    uint2 pick[32];
  } few;
  struct {
    union {
      double s64[RT_EMAX];  // scores by expert, then group scores
      struct {
        float s[RT_EMAX], score[RT_EMAX];
      };
    };
    int keep[RT_EMAX];
  } group;
};

// A group's score of its best scores: one that lacks a second expert ranks at -inf, also
// where the first one's is +inf.
template <typename F>
__device__ __forceinline__ F group_score(const RouteArgs& a, F b1, F b2) {
  if (a.group_top == 1) return b1;
  return b2 == -INFINITY ? b2 : b1 + b2;
}

// A token in 64 bits: the definition itself, in little code rather than little time.
template <typename LT>
__device__ __noinline__ void route_token_f64(const RouteArgs& a, int64_t t, RouteShared& sh) {
  const int lane = threadIdx.x & 31;
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  double* key = sh.f64;
  // of expert e, lane e % 32's
  float m = -INFINITY;
  for (int e = lane; e < a.E; e += 32) m = fmaxf(m, load1(row + e));
  m = warp_max(m);
  // affinities; a logit of -inf takes its expert out, also where all are -inf
  auto affinity = [&](int e) {
    const double x = load1(row + e);
    if (x == -INFINITY) return 0.0;
    const double v = exp(a.softmax ? x - (double)m : -x);
    return a.softmax ? v : 1.0 / (1.0 + v);
  };
  double z = 0.0;
  __syncwarp();
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    const double p = affinity(e);
    key[e] = p;
    z += p;
  }
  z = warp_sum(z);
  const double rz = z == 0.0 ? 0.0 : 1.0 / z, unit = a.softmax ? rz : 1.0;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    const double p = key[e];
    if (a.probs) a.probs[t * a.E + e] = (float)(p * rz);
    double s = p * unit + (a.bias ? (double)a.bias[e] : 0.0);
    if (load1(row + e) == -INFINITY || s != s) s = -INFINITY;
    key[e] = s;
  }
  __syncwarp();
  uint32_t out = 0;  // experts (lane + 32 i in bit i) of groups that are not kept
  if (a.n_group > 1) {
    const int size = a.E / a.n_group;
    double* of_group = sh.f64 + RT_EMAX;
#pragma unroll 1
    for (int g = lane; g < a.n_group; g += 32) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const double v = key[g * size + i];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
      of_group[g] = group_score(a, b1, b2);
    }
    __syncwarp();
#pragma unroll 1
    for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
      const int g = e / size;
      const double mine = of_group[g];
      int before = 0;
      for (int h = 0; h < a.n_group; ++h) {
        const double v = of_group[h];
        before += v > mine || (v == mine && h < g);
      }
      out |= (before >= a.topk_group ? 1u : 0u) << i;
    }
    __syncwarp();
  }
#pragma unroll 1
  for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
    // without a bias the logits rank the experts: the same order, and no rounding in it
    const float x = load1(row + e);
    if (a.bias == nullptr && key[e] != -INFINITY) key[e] = x;
    if (x != x && a.bias == nullptr) key[e] = -INFINITY;
    if (out >> i & 1) key[e] = -INFINITY;
  }
  uint32_t picked = 0;  // as out
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int at = RT_EMAX;
    for (int e = lane, i = 0; e < a.E; e += 32, ++i)
      if (!(picked >> i & 1) && (at == RT_EMAX || key[e] > best)) {
        best = key[e];
        at = e;
      }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      const double v = __shfl_xor_sync(FULL, best, o);
      const int e = __shfl_xor_sync(FULL, at, o);
      if (e != RT_EMAX && (at == RT_EMAX || v > best || (v == best && e < at))) {
        best = v;
        at = e;
      }
    }
    if ((at & 31) == lane) picked |= 1u << (at >> 5);
    if (lane == 0) a.idx[t * a.k + j] = at;
  }
  __syncwarp();  // idx is there for every lane
  auto weight = [&](int j) {
    const int e = a.idx[t * a.k + j];
    const double p = affinity(e) * unit;
    return key[e] == -INFINITY && p == p ? 0.0 : p;  // 0: nothing was left to choose from
  };
  double sum = 0.0;
#pragma unroll 1
  for (int j = lane; j < a.k; j += 32) sum += weight(j);
  sum = warp_sum(sum);
  const double f = a.renorm ? (sum == 0.0 ? 0.0 : a.scale / sum) : (double)a.scale;
#pragma unroll 1
  for (int j = lane; j < a.k; j += 32) a.w[t * a.k + j] = (float)(weight(j) * f);
}

// 1 / v to two steps of FP32 (0 for an infinite v).
__device__ __forceinline__ float quick_rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Affinities and scores are computed by operations that are never contracted: equal logits
// and biases give equal bits wherever they stand, so that their order is that of the experts.
template <bool SOFT>
__device__ __forceinline__ float affinity(float x, float m) {
  return SOFT ? expf(x - m) : quick_rcp(__fadd_rn(1.0f, expf(-x)));
}

// A lane's best values, descending: all of them, or the best four.
template <int EPL>
struct Best {
  static constexpr int N = EPL < 4 ? EPL : 4;
  uint32_t v[N];

  __device__ __forceinline__ static void order(uint32_t& hi, uint32_t& lo) {
    const uint32_t h = max(hi, lo);
    lo = min(hi, lo);
    hi = h;
  }
  __device__ __forceinline__ static void sort4(uint32_t* a) {
    order(a[0], a[1]);
    order(a[2], a[3]);
    order(a[0], a[2]);
    order(a[1], a[3]);
    order(a[1], a[2]);
  }
  __device__ __forceinline__ void of(const uint32_t (&u)[EPL]) {
    uint32_t a[EPL];
#pragma unroll
    for (int q = 0; q < EPL; ++q) a[q] = u[q];
    if constexpr (EPL == 2) {
      order(a[0], a[1]);
    } else {
      sort4(a);
#pragma unroll
      for (int n = 4; n < EPL; n += 4) {
        // the larger half of two descending fours, then in order
        sort4(a + n);
#pragma unroll
        for (int q = 0; q < 4; ++q) a[q] = max(a[q], a[n + 3 - q]);
        order(a[0], a[2]);
        order(a[1], a[3]);
        order(a[0], a[1]);
        order(a[2], a[3]);
      }
    }
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = a[q];
  }
  // The best of u once all of v are taken: `last` was the lowest of them.
  __device__ __forceinline__ void refill(uint32_t (&u)[EPL], uint32_t last) {
    int same = N;  // of v, equal to the last
#pragma unroll
    for (int q = 0; q < EPL; ++q) same -= u[q] > last;
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if (u[q] > last || (u[q] == last && same-- > 0)) u[q] = 0;
    of(u);
  }
  __device__ __forceinline__ void pop() {
#pragma unroll
    for (int q = 0; q + 1 < N; ++q) v[q] = v[q + 1];
    v[N - 1] = 0;
  }
};

// Which groups stay, in 64 bits where FP32 does not settle it: a group's lanes share its
// experts (one lane a group where there are more than 16).
template <typename LT>
__device__ __noinline__ void refine_groups(const RouteArgs& a, const LT* row, float m,
                                           RouteShared& sh) {
  const int lane = threadIdx.x & 31, size = a.E / a.n_group;
  double z = 0.0, rz = 1.0;
  __syncwarp();
#pragma unroll 2
  for (int e = lane; e < a.E; e += 32) {
    const double x = load1(row + e), v = exp(a.softmax ? x - (double)m : -x);
    const double p = a.softmax ? v : 1.0 / (1.0 + v);
    sh.group.s64[e] = p;
    z += p;
  }
  if (a.softmax) rz = 1.0 / warp_sum(z);
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    const double s = sh.group.s64[e] * rz + (a.bias ? (double)a.bias[e] : 0.0);
    sh.group.s64[e] = load1(row + e) == -INFINITY || s != s ? -INFINITY : s;
  }
  __syncwarp();
  int share = 1;  // lanes of a group
  while (share * 2 * a.n_group <= 32) share *= 2;
  const int at = lane & (share - 1);
  double score[RT_EMAX / 32];  // of this lane's groups
#pragma unroll
  for (int i = 0; i < RT_EMAX / 32; ++i) {
    const int g = lane / share + i * (32 / share);
    if (i * 32 >= a.n_group * share) break;
    double b1 = -INFINITY, b2 = -INFINITY;
    if (g < a.n_group)
#pragma unroll 4
      for (int n = at; n < size; n += share) {
        const double v = sh.group.s64[g * size + n];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
    for (int o = 1; o < share; o <<= 1) {
      const double o1 = __shfl_xor_sync(FULL, b1, o), o2 = __shfl_xor_sync(FULL, b2, o);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    score[i] = group_score(a, b1, b2);
  }
  __syncwarp();
  double* of_group = sh.group.s64;
#pragma unroll
  for (int i = 0; i < RT_EMAX / 32; ++i) {
    const int g = lane / share + i * (32 / share);
    if (at == 0 && g < a.n_group && i * 32 < a.n_group * share) of_group[g] = score[i];
  }
  __syncwarp();
#pragma unroll 1
  for (int g = lane; g < a.n_group; g += 32) {
    const double mine = of_group[g];
    int before = 0;
#pragma unroll 4
    for (int h = 0; h < a.n_group; ++h) {
      const double v = of_group[h];
      before += v > mine || (v == mine && h < g);
    }
    sh.group.keep[g] = before < a.topk_group;
  }
}

// The error of a group's score, of its best scores b1 and b2: an affinity's error and a rounding
// for each of its terms, and its own.  NaN where the sum of two finite scores leaves FP32.
__device__ __forceinline__ float group_error(const RouteArgs& a, float b1, float b2,
                                             float two_dp) {
  const float m1 = fabsf(b1), m2 = a.group_top == 2 ? fabsf(b2) : 0.0f;
  if (m1 + m2 < INFINITY) return two_dp + 0x1p-22f * (m1 + m2);
  return fmaxf(m1, m2) < INFINITY ? NAN : two_dp;
}

// Gives the experts of groups that are not kept the score -inf.  two_dp: twice an
// affinity's error; m: the largest logit, for refine_groups.
template <typename LT, int EPL>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, const LT* row, float m,
                                            RouteShared& sh, float (&s)[EPL], float two_dp) {
  const int lane = threadIdx.x & 31, e0 = lane * EPL;
  const int size = a.E / a.n_group, lanes = size / EPL;
  // of the groups that this lane compares, ordered: the lowest score kept, less its error,
  // and the highest that is not, and its error
  uint32_t low = 0xffffffffu, high = 0;
  float err = 0.0f;
  auto score = [&](float b1, float b2) {
    err = group_error(a, b1, b2, two_dp);
    return group_score(a, b1, b2);
  };
  auto clear = [&]() {
    const float lo = unordered(__reduce_min_sync(FULL, low));
    const uint32_t most = __reduce_max_sync(FULL, high);
    return lo > unordered(most) || most <= ORD_NEG_INF;
  };
  auto sort_out = [&](float mine, bool keep) {
    if (keep) low = min(low, ordered(mine - err));
    else high = max(high, ordered(mine + err));
    if (err != err) high = 0xffffffffu;
  };
  if (lanes * EPL == size && (lanes & (lanes - 1)) == 0) {  // a group is 1, 2, ... 32 lanes
    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      b2 = fmaxf(b2, fminf(b1, s[q]));
      b1 = fmaxf(b1, s[q]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const float o1 = __shfl_xor_sync(FULL, b1, o), o2 = __shfl_xor_sync(FULL, b2, o);
      b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
      b1 = fmaxf(b1, o1);
    }
    const float mine = e0 < a.E ? score(b1, b2) : -INFINITY;
    // the lanes of a group share the comparison with the others
    const int at = lane & -lanes;  // the group's first lane
    int before = 0;
    for (int h = 0; h < a.n_group; h += lanes) {
      const int o = (h + lane - at) * lanes;  // the other group's first lane
      const float v = __shfl_sync(FULL, mine, o & 31);
      before += (v > mine || (v == mine && o < at)) && h + lane - at < a.n_group;
    }
    for (int o = 1; o < lanes; o <<= 1) before += __shfl_xor_sync(FULL, before, o);
    const bool keep = before < a.topk_group;
    if (e0 < a.E) sort_out(mine, keep);
    if (clear()) {
      if (!keep) {
#pragma unroll
        for (int q = 0; q < EPL; ++q) s[q] = -INFINITY;
      }
      return;
    }
    refine_groups(a, row, m, sh);
  } else {
    // lane g % 32 looks after group g
    float* all = sh.group.s;
    float* of_group = sh.group.score;
    constexpr int MOST = RT_EMAX / 32;
    float mine[MOST], off[MOST];
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if (e0 + q < a.E) all[e0 + q] = s[q];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      const int g = lane + 32 * i;
      if (g >= a.n_group) break;
      float b1 = -INFINITY, b2 = -INFINITY;
      for (int n = 0; n < size; ++n) {
        const float v = all[g * size + n];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
      of_group[g] = mine[i] = score(b1, b2);
      off[i] = err;
    }
    __syncwarp();
    uint32_t kept = 0;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      const int g = lane + 32 * i;
      if (g >= a.n_group) break;
      int before = 0;
      for (int h = 0; h < a.n_group; ++h) {
        const float v = of_group[h];
        before += v > mine[i] || (v == mine[i] && h < g);
      }
      err = off[i];
      sort_out(mine[i], before < a.topk_group);
      kept |= (before < a.topk_group ? 1u : 0u) << i;
    }
    __syncwarp();
    if (clear()) {
#pragma unroll
      for (int i = 0; i < MOST; ++i)
        if (lane + 32 * i < a.n_group) sh.group.keep[lane + 32 * i] = kept >> i & 1;
    } else {
      refine_groups(a, row, m, sh);
    }
  }
  __syncwarp();
  int g = e0 / size, left = size - (e0 - g * size);  // the next expert's group
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    if (e0 + q < a.E && !sh.group.keep[g]) s[q] = -INFINITY;
    if (--left == 0) {
      left = size;
      ++g;
    }
  }
  __syncwarp();
}

// 1 / sum of a softmax's terms, in 64 bits.
template <typename LT>
__device__ __noinline__ double rz_f64(const LT* row, int E, float m) {
  double z = 0.0;
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < E; e += 32) z += exp((double)load1(row + e) - (double)m);
  return 1.0 / warp_sum(z);
}

// The lowest key whose score may be the last pick's: within twice an affinity's error and the
// scores' own roundings of it.  A score of +inf has neither, and what ranks at -inf (taken out,
// or of a group that is not kept) is not in question beside the lowest finite score either.
__device__ __forceinline__ uint32_t lowest_near(uint32_t last, float two_dp) {
  const float s = unordered(last);
  if (s == INFINITY) return last;
  return max(ordered(s - (two_dp + 0x1p-22f * fabsf(s))), ORD_NEG_INF + 1);
}

// The picks of a token where FP32 does not settle their order, after route_token and its
// outputs: among the experts whose keys are `least` or more, one a lane, by 64-bit scores.
// The token's SEG lanes from `base` on hold EPL experts each, by slot in keys and ps;
// list [64] is free.  For a softmax 1 / z is at first still FP32's rz, off by 25 u of itself,
// which moves the difference of two scores by 25 u times that of their affinities; where that
// is too much, z is summed in 64 bits too.  False where the token needs 64 bits as a whole.
template <typename LT, int SEG, int EPL>
__device__ __noinline__ bool refine(const RouteArgs& a, int64_t t, float m, float rz,
                                    uint32_t least, const uint32_t* keys, const float* ps,
                                    int base, int* list) {
  const int lane = threadIdx.x & 31, l = lane - base;
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  const bool has = l >= 0 && l < SEG;
  uint32_t u[EPL], bits = 0;
  get(keys, lane, u);
#pragma unroll
  for (int q = 0; q < EPL; ++q) bits |= (has && u[q] >= least ? 1u : 0u) << q;
  const int mine = __popc(bits);
  int at = mine;  // those up to this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL, at, o);
    if (lane >= o) at += v;
  }
  const int n = __shfl_sync(FULL, at, 31);
  if (n == 0 || n > 32) return false;  // every lane below reads an entry of the list
  at -= mine;
  __syncwarp();
  for (; bits; bits &= bits - 1) list[at++] = l * EPL + __ffs(bits) - 1;
  __syncwarp();
  const int c = list[lane < n ? lane : 0];
  const float b = a.bias[c];
  const double x = load1(row + c), v = exp(a.softmax ? x - (double)m : -x);
  int rank = 0;
  bool sure = a.softmax;
  if (a.softmax) {
    const double p = v * rz;
    for (int h = 0; h < n; ++h) {
      const double dp = __shfl_sync(FULL, p, h) - p, bh = __shfl_sync(FULL, b, h);
      const double ds = dp + (bh - b);
      rank += ds > 0.0 || (ds == 0.0 && h < lane);
      // 64 u of the affinities' difference, and the scores' own rounding in 64 bits
      sure &= fabs(ds) > 0x1p-18 * fabs(dp) + 0x1p-50 * (fabs(bh) + 1.0) || (dp == 0.0 && bh == b);
    }
    sure = __all_sync(FULL, sure || lane >= n);
  }
  if (!sure) {
    const double s = (a.softmax ? v * rz_f64(row, a.E, m) : 1.0 / (1.0 + v)) + (double)b;
    rank = 0;
    for (int h = 0; h < n; ++h) {
      const double o = __shfl_sync(FULL, s, h);
      rank += o > s || (o == s && h < lane);
    }
  }
  // pick `rank` and its weight; picks from n on are those that rank at -inf, already there
  const bool pick = lane < n && rank < a.k;
  const float p = pick ? ps[slot<EPL>(base + c / EPL, c % EPL)] : 0.0f;
  const float sum = warp_sum(p);
  if (!(sum > RT_SMALL_SUM) || __any_sync(FULL, pick && p < RT_TINY)) return false;
  if (pick) {
    const float f = a.renorm ? quick_rcp(sum) : a.softmax ? rz : 1.0f;
    a.idx[t * a.k + rank] = c;
    a.w[t * a.k + rank] = a.scale * (p * f);
  }
  return true;
}

enum { RT_DONE, RT_NEAR, RT_STOP };

// A token in 32 bits: RT_STOP where that does not give the weights, RT_NEAR where it may not
// give the picks' order, which is then refine's work with what `near` holds.
struct Near {
  float m, rz;     // the largest logit (0 for sigmoids), 1 / z
  uint32_t least;  // lowest key in question
};
//
// Errors, with u = 2^-24: expf and the quick reciprocal are off by 2 u of their values.
//   sigmoid  p = 1 / (1 + e): u (2 (1 - p) + 1 + 2) p <= 3 u
//   softmax  x - m by |x - m| u, so e by (|x - m| + 2) u; z, a sum of positive terms over
//            at most 12 additions, by (12 + 2 + sum p |x - m|) u with that sum at most
//            ln 256 (the entropy's bound); 1 / z by 2 u, the product by u.  Together at most
//            p (|x - m| + 25) u <= 25 u max p, the largest where x = m.
// Twice that is 6 u and 50 u / z; the margins take 8 u and 64 u / z.  Adding the bias rounds
// by u |score|; 2 u a score stand in the margin.
template <typename LT, int EPL, bool SOFT, bool VEC, bool GROUPS>
__device__ __forceinline__ int route_token(const RouteArgs& a, int64_t t, RouteShared& sh,
                                           Near& question) {
  const int lane = threadIdx.x & 31, e0 = lane * EPL;
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  const bool bias = a.bias != nullptr;
  auto here = [&](int q) { return VEC ? e0 < a.E : e0 + q < a.E; };
  float x[EPL], b[EPL];
  load_row(x, row, e0, a.E, VEC, -INFINITY);
  if (bias) load_row(b, a.bias, e0, a.E, VEC, 0.0f);
  float m = 0.0f;
  if (SOFT) {
    m = x[0];
#pragma unroll
    for (int q = 1; q < EPL; ++q) m = fmaxf(m, x[q]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;
  }
  float p[EPL], z = 0.0f;
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    p[q] = affinity<SOFT>(x[q], m);  // 0 for a logit of -inf
    z += p[q];
  }
  z = warp_sum(z);
  if (!(z > RT_SMALL_ALL)) return RT_STOP;  // nearly nothing, nothing, or a NaN
  const float rz = quick_rcp(z);
  float s[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) s[q] = __fmul_rn(p[q], rz);
  if (a.probs) store_row(a.probs + t * a.E, s, e0, a.E, VEC);
  const float two_dp = SOFT ? 0x1p-18f * rz : 0x1p-21f;
  // scores; without a bias the logits rank the experts, exactly
  if (bias || GROUPS) {
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      if (!SOFT) s[q] = p[q];
      if (bias) s[q] = fmaxf(__fadd_rn(s[q], b[q]), -INFINITY);  // a NaN ranks as -inf
      if (x[q] == -INFINITY) s[q] = -INFINITY;
    }
    if constexpr (GROUPS) keep_groups(a, row, m, sh, s, two_dp);
  }
  if (!bias) {
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if (!GROUPS || s[q] != -INFINITY) s[q] = x[q];
  }
  uint32_t u[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    u[q] = here(q) ? ordered(s[q]) : 0;
  }
  put(sh.f32.key, lane, u);
  put(sh.f32.p, lane, p);
  Best<EPL> best;
  best.of(u);
  // pick j and its lane go to lane j: picks[j] in shared memory
  uint32_t last = 0, gone = 0;  // gone: of this lane's best
  const uint32_t lower = (1u << lane) - 1;
  for (int j = 0; j < a.k; ++j) {
    last = __reduce_max_sync(FULL, best.v[0]);
    const uint32_t has = __ballot_sync(FULL, best.v[0] == last);
    const bool win = best.v[0] == last && (has & lower) == 0;
    if (win) {
      sh.f32.pick[j] = make_uint2(last, lane);
      best.pop();
      ++gone;
    }
    if constexpr (Best<EPL>::N < EPL) {
      if (__any_sync(FULL, gone == Best<EPL>::N) && gone == Best<EPL>::N) {
        best.refill(u, last);
        gone = 0;
      }
    }
  }
  __syncwarp();  // the picks, the keys and the affinities are in shared memory
  // which expert: the n-th of lane src's with this key, n picks of the same key before it
  const bool mine = lane < a.k;
  const uint2 pick = mine ? sh.f32.pick[lane] : make_uint2(0, 0);
  const uint32_t key = pick.x;
  const int src = (int)pick.y;
  const uint32_t up_key = __shfl_up_sync(FULL, key, 1);
  const int up_src = __shfl_up_sync(FULL, src, 1);
  uint32_t where = 0;
  get(sh.f32.key, src, u);
#pragma unroll
  for (int q = 0; q < EPL; ++q) where |= (u[q] == key ? 1u : 0u) << q;
  if (__any_sync(FULL, mine && lane > 0 && key == up_key && src == up_src)) {
    const unsigned long long id = mine ? (unsigned long long)key << 6 | src : 32 + lane;
    int n = __popc(__match_any_sync(FULL, id) & lower);
    for (; n > 0; --n) where &= where - 1;
  }
  const int e = mine ? src * EPL + __ffs(where) - 1 : 0;
  bool near = false;
  if (bias) {
    const uint32_t down = __shfl_down_sync(FULL, key, 1);
    const float sc = unordered(key), dn = unordered(down);
    near = lane + 1 < a.k && down != ORD_NEG_INF &&
                !(sc - dn > two_dp + 0x1p-23f * (fabsf(sc) + fabsf(dn)));
    if (__any_sync(FULL, near)) {  // equal in 64 bits too?
      const int en = __shfl_down_sync(FULL, e, 1);
      near = near && !(load1(row + e) == load1(row + en) && a.bias[e] == a.bias[en] && e < en);
    }
    // and the first that is not picked
    const uint32_t after = __reduce_max_sync(FULL, best.v[0]);
    const uint32_t least = lowest_near(last, two_dp);
    if (after > ORD_NEG_INF && after >= least) {  // equal in 64 bits too?
      const int el = __shfl_sync(FULL, e, a.k - 1);
      const float xl = load1(row + el), bl = a.bias[el];
      get(sh.f32.key, lane, u);
#pragma unroll
      for (int q = 0; q < EPL; ++q)
        if (u[q] >= least && u[q] <= last)
          near |= !(u[q] == last && load1(row + e0 + q) == xl && a.bias[e0 + q] == bl);
    }
    question = {m, rz, least};
  }
  const bool some = mine && key != ORD_NEG_INF;  // not: nothing was left to choose from
  const float pe = some ? sh.f32.p[slot<EPL>(e / EPL, e % EPL)] : 0.0f;
  const float sum = warp_sum(pe);
  bool bad = some && !(sum > RT_SMALL_SUM);
  if (some && pe < RT_TINY) bad |= load1(row + e) - m > -140.0f;
  if (__any_sync(FULL, bad)) return RT_STOP;
  if (mine) {
    const float f = a.renorm ? (sum == 0.0f ? 0.0f : quick_rcp(sum)) : (SOFT ? rz : 1.0f);
    a.idx[t * a.k + lane] = e;
    a.w[t * a.k + lane] = a.scale * (pe * f);
  }
  return __any_sync(FULL, near) ? RT_NEAR : RT_DONE;
}

// route_token and what its answer asks for; sh.f32 is by slots of EPL experts a lane.
template <typename LT, int EPL, bool SOFT, bool VEC, bool GROUPS>
__device__ __forceinline__ void route_whole(const RouteArgs& a, int64_t t, RouteShared& sh) {
  Near q;
  const int rc = route_token<LT, EPL, SOFT, VEC, GROUPS>(a, t, sh, q);
  if (rc == RT_DONE) return;
  if (rc == RT_NEAR) {
    __syncwarp();
    if (refine<LT, 32, EPL>(a, t, q.m, q.rz, q.least, sh.f32.key, sh.f32.p, 0,
                            reinterpret_cast<int*>(sh.f32.pick)))
      return;
  }
  __syncwarp();
  route_token_f64<LT>(a, t, sh);
}

// A warp a token: a loop over tokens with the next one's logits on their way took 1.5 times
// as long, since its state does not fit the registers beside the calls.
template <typename LT, int EPL, bool SOFT, bool VEC, bool GROUPS>
__global__ void __launch_bounds__(RT_WARPS * 32, EPL == 8 ? 8 : 10)
    route_topk_kernel(const RouteArgs a) {
  __shared__ __align__(16) RouteShared sh[RT_WARPS];
  behind();
  const int warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp;
  if (t >= a.T) return;
  // lane j looks after pick j: more than 32 picks take the 64-bit way
  if (a.k > 32) route_token_f64<LT>(a, t, sh[warp]);
  else route_whole<LT, EPL, SOFT, VEC, GROUPS>(a, t, sh[warp]);
}

// ---- several tokens a warp
// Where there are tokens enough to fill the SMs, a token takes SEG lanes of EPL experts, and
// the 32 / SEG tokens of a warp share the instructions of the picks, sums and checks (480 a
// token with a warp each, 128 experts and 6 picks).  The steps are route_token's; a token
// that its checks stop is done again by the whole warp.

template <int SEG>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int o = 1; o < SEG; o <<= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
template <int SEG>
__device__ __forceinline__ uint32_t seg_max(uint32_t v) {
#pragma unroll
  for (int o = 1; o < SEG; o <<= 1) v = max(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
// Sum of a lane's values, in pairs: log2(N) roundings.
template <int N>
__device__ __forceinline__ float pair_sum(const float (&v)[N]) {
  float t[N];
#pragma unroll
  for (int q = 0; q < N; ++q) t[q] = v[q];
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
    for (int q = 0; q < n; ++q) t[q] += t[q + n];
  return t[0];
}

template <typename LT, int EPL, bool SOFT, bool GROUPS>
__device__ __noinline__ void route_token_again(const RouteArgs& a, int64_t t, RouteShared& sh) {
  route_whole<LT, EPL, SOFT, true, GROUPS>(a, t, sh);
}

template <typename LT, int SEG, int EPL, bool SOFT, bool GROUPS>
__global__ void __launch_bounds__(RT_WARPS * 32, 8)
    route_topk_few_kernel(const RouteArgs a) {
  constexpr int TOKENS = 32 / SEG;
  constexpr uint32_t ALL = (1u << SEG) - 1;  // lanes of a segment
  __shared__ __align__(16) RouteShared shared[RT_WARPS];
  behind();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  RouteShared& sh = shared[warp];
  const int64_t t0 = ((int64_t)blockIdx.x * RT_WARPS + warp) * TOKENS;
  if (t0 >= a.T) return;
  const int l = lane & (SEG - 1), base = lane - l, e0 = l * EPL;
  const bool real = t0 + lane / SEG < a.T, here = e0 < a.E;
  const int64_t t = real ? t0 + lane / SEG : a.T - 1;
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  const bool bias = a.bias != nullptr;
  float x[EPL];
  load_row(x, row, e0, a.E, true, -INFINITY);
  float m = 0.0f;
  if (SOFT) {
    m = x[0];
#pragma unroll
    for (int q = 1; q < EPL; ++q) m = fmaxf(m, x[q]);
#pragma unroll
    for (int o = 1; o < SEG; o <<= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    if (m == -INFINITY) m = 0.0f;
  }
  float p[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) p[q] = affinity<SOFT>(x[q], m);
  const float z = seg_sum<SEG>(pair_sum(p));
  bool bad = !(z > RT_SMALL_ALL);
  const float rz = quick_rcp(z);
  put(sh.few.p, lane, p);
  float s[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) s[q] = __fmul_rn(p[q], rz);
  if (a.probs && real) store_row(a.probs + t * a.E, s, e0, a.E, true);
  const float two_dp = SOFT ? 0x1p-18f * rz : 0x1p-21f;
  if (bias || GROUPS) {
    float b[EPL];
    if (bias) load_row(b, a.bias, e0, a.E, true, 0.0f);
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      if (!SOFT) s[q] = p[q];
      if (bias) s[q] = fmaxf(__fadd_rn(s[q], b[q]), -INFINITY);
      if (x[q] == -INFINITY) s[q] = -INFINITY;
    }
  }
  bool out = false;  // the lane's group does not stay
  if (GROUPS) {      // a group is 1, 2, 4, ... lanes
    const int lanes = a.E / a.n_group / EPL;
    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      b2 = fmaxf(b2, fminf(b1, s[q]));
      b1 = fmaxf(b1, s[q]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const float o1 = __shfl_xor_sync(FULL, b1, o), o2 = __shfl_xor_sync(FULL, b2, o);
      b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
      b1 = fmaxf(b1, o1);
    }
    const float err = group_error(a, b1, b2, two_dp);
    const float mine = group_score(a, b1, b2);
    const int at = l & -lanes;
    int before = 0;
    for (int h = 0; h < a.n_group; h += lanes) {
      const int o = (h + l - at) * lanes;
      const float v = __shfl_sync(FULL, mine, base + (o & (SEG - 1)));
      before += (v > mine || (v == mine && o < at)) && h + l - at < a.n_group;
    }
    for (int o = 1; o < lanes; o <<= 1) before += __shfl_xor_sync(FULL, before, o);
    out = before >= a.topk_group;
    // ~low: the lowest score kept, as a maximum
    uint32_t low = here && !out ? ~ordered(mine - err) : 0;
    uint32_t high = here && out ? ordered(mine + err) : 0;
    low = ~seg_max<SEG>(low);
    high = seg_max<SEG>(high);
    bad |= (here && err != err) || !(unordered(low) > unordered(high) || high <= ORD_NEG_INF);
  }
  uint32_t u[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    if (!bias) s[q] = x[q];
    if (GROUPS && out) s[q] = -INFINITY;
    u[q] = here ? ordered(s[q]) : 0;
  }
  put(sh.few.key, lane, u);
  Best<EPL> best;
  best.of(u);
  uint32_t last = 0, gone = 0;
  const uint32_t lower = ((1u << lane) - 1) & ALL << base;  // the segment's lanes before this
  for (int j = 0; j < a.k; ++j) {
    last = seg_max<SEG>(best.v[0]);
    const bool has = best.v[0] == last;
    const uint32_t those = __ballot_sync(FULL, has);
    if (has && (those & lower) == 0) {
      sh.few.pick[base + j] = make_uint2(last, lane);
      best.pop();
      ++gone;
    }
    if constexpr (Best<EPL>::N < EPL) {
      if (__any_sync(FULL, gone == Best<EPL>::N) && gone == Best<EPL>::N) {
        best.refill(u, last);
        gone = 0;
      }
    }
  }
  __syncwarp();
  // lane j of the segment looks after pick j
  const bool mine = l < a.k;
  const uint2 pick = mine ? sh.few.pick[lane] : make_uint2(0, lane);
  const uint32_t key = pick.x;
  const int src = (int)pick.y;
  const uint32_t up_key = __shfl_up_sync(FULL, key, 1);
  const int up_src = __shfl_up_sync(FULL, src, 1);
  uint32_t where = 0;
  get(sh.few.key, src, u);
#pragma unroll
  for (int q = 0; q < EPL; ++q) where |= (u[q] == key ? 1u : 0u) << q;
  if (__any_sync(FULL, mine && l > 0 && key == up_key && src == up_src)) {
    const unsigned long long id = mine ? (unsigned long long)key << 6 | src : 32 + lane;
    int n = __popc(__match_any_sync(FULL, id) & ((1u << lane) - 1));
    for (; n > 0; --n) where &= where - 1;
  }
  const int e = mine ? (src - base) * EPL + __ffs(where) - 1 : 0;
  bool near = false;
  uint32_t least = 0;
  if (bias) {
    const uint32_t down = __shfl_down_sync(FULL, key, 1);
    const float sc = unordered(key), dn = unordered(down);
    near = l + 1 < a.k && down != ORD_NEG_INF &&
                !(sc - dn > two_dp + 0x1p-23f * (fabsf(sc) + fabsf(dn)));
    if (__any_sync(FULL, near)) {  // equal in 64 bits too?
      const int en = __shfl_down_sync(FULL, e, 1);
      near = near && !(load1(row + e) == load1(row + en) && a.bias[e] == a.bias[en] && e < en);
    }
    const uint32_t after = seg_max<SEG>(best.v[0]);
    least = lowest_near(last, two_dp);
    const bool close = after > ORD_NEG_INF && after >= least;
    if (__any_sync(FULL, close)) {  // equal in 64 bits too?
      const int el = __shfl_sync(FULL, e, base + a.k - 1);
      if (close) {
        const float xl = load1(row + el), bl = a.bias[el];
        get(sh.few.key, lane, u);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (u[i] >= least && u[i] <= last)
            near |= !(u[i] == last && load1(row + e0 + i) == xl && a.bias[e0 + i] == bl);
      }
    }
  }
  const bool some = mine && key != ORD_NEG_INF;
  const float pe = some ? sh.few.p[slot<EPL>(base + e / EPL, e % EPL)] : 0.0f;
  const float sum = seg_sum<SEG>(pe);
  bad |= some && !(sum > RT_SMALL_SUM);
  if (some && pe < RT_TINY) bad |= load1(row + e) - m > -140.0f;
  const uint32_t stopped = __ballot_sync(FULL, bad && real);
  if (mine && real && !(stopped & ALL << base)) {
    const float f = a.renorm ? (sum == 0.0f ? 0.0f : quick_rcp(sum)) : (SOFT ? rz : 1.0f);
    a.idx[t * a.k + l] = e;
    a.w[t * a.k + l] = a.scale * (pe * f);
  }
  const uint32_t nears = __ballot_sync(FULL, near && real);
  if ((stopped | nears) == 0) return;
  uint32_t again = stopped;
  for (int i = 0; i < TOKENS; ++i)
    if (nears >> (i * SEG) & ~stopped >> (i * SEG) & ALL) {
      const int from = i * SEG;
      __syncwarp();
      if (!refine<LT, SEG, EPL>(a, t0 + i, __shfl_sync(FULL, m, from), __shfl_sync(FULL, rz, from),
                                __shfl_sync(FULL, least, from), sh.few.key, sh.few.p, from,
                                reinterpret_cast<int*>(sh.few.pick)))
        again |= 1u << from;
    }
  for (int i = 0; i < TOKENS; ++i)
    if (again >> (i * SEG) & ALL) {
      __syncwarp();  // sh and probs are free
      route_token_again<LT, SEG * EPL / 32, SOFT, GROUPS>(a, t0 + i, sh);
    }
}

struct RouteBwdArgs {
  const void* logits;
  const int32_t* idx;
  const float *w, *dw, *seq_grad;
  void* dlogits;
  int64_t T, seq_len;
  int E, k, renorm, softmax;
  int vec, few;  // as in RouteArgs, of logits, seq_grad and dlogits
  float scale;
};

// A token's gradient in 64 bits, in little code rather than little time.  dp: [E] in
// shared memory.
template <typename LT>
__device__ __noinline__ void route_bwd_f64(const RouteBwdArgs& a, int64_t t, double* dp) {
  const int lane = threadIdx.x & 31;
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  float m = -INFINITY;
  for (int e = lane; e < a.E; e += 32) m = fmaxf(m, load1(row + e));
  m = warp_max(m);
  double unit = 1.0;  // of p
  auto affinity = [&](int e) {
    const double x = load1(row + e);
    if (x == -INFINITY) return 0.0;
    const double v = exp(a.softmax ? x - (double)m : -x);
    return a.softmax ? v * unit : 1.0 / (1.0 + v);
  };
  double z = 0.0;
  __syncwarp();
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    z += affinity(e);
    dp[e] = 0.0;
  }
  z = warp_sum(z);
  const double rz = z == 0.0 ? 0.0 : 1.0 / z;
  if (a.softmax) unit = rz;
  // the picks: their affinities' sum and the gradients' product with the weights
  auto counts = [&](int j) {
    const int e = a.idx[t * a.k + j];
    return a.w[t * a.k + j] != 0.0f && e >= 0 && e < a.E;
  };
  double zc = 0.0, dot = 0.0;
#pragma unroll 1
  for (int j = lane; j < a.k; j += 32)
    if (counts(j)) {
      dot += (double)a.dw[t * a.k + j] * a.w[t * a.k + j];
      zc += affinity(a.idx[t * a.k + j]);
    }
  zc = warp_sum(zc);
  dot = warp_sum(dot);
  const double rzc = a.renorm ? 1.0 / zc : 1.0;
  if (!a.renorm) dot = 0.0;
  __syncwarp();
#pragma unroll 1
  for (int j = 0; j < a.k; ++j)  // one after another: an expert may stand there twice
    if (counts(j) && lane == (a.idx[t * a.k + j] & 31))
      dp[a.idx[t * a.k + j]] += ((double)a.scale * a.dw[t * a.k + j] - dot) * rzc;
  const float* g = a.seq_grad ? a.seq_grad + (t / a.seq_len) * a.E : nullptr;
  double cg = 0.0, c = 0.0;
  if (g && !a.softmax) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) cg += affinity(e) * rz * g[e];
    cg = warp_sum(cg);
  }
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    double d = dp[e];
    if (g) d += a.softmax ? (double)g[e] : (g[e] - cg) * rz;
    dp[e] = d;
    if (a.softmax) c += affinity(e) * d;
  }
  c = warp_sum(c);
  LT* out = reinterpret_cast<LT*>(a.dlogits) + t * a.E;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    double v;
    if (a.softmax) {
      v = affinity(e) * (dp[e] - c);
    } else {  // p (1 - p) without the cancellation of 1 - p
      const double h = exp(-fabs((double)load1(row + e)));
      v = dp[e] * (h / ((1.0 + h) * (1.0 + h)));
    }
    store1(out + e, (float)v);
  }
}

// A token takes SEG lanes of EPL experts, as in the forward, and has at most SEG picks, lane
// j of them looking after pick j.  What bounds it is latency, so the sums run side by side:
// a softmax's sum of p dp over the picks comes from that of p dw.  Tokens whose affinities
// leave FP32's range, or with more picks, are done in 64 bits.
template <typename LT, int SEG, int EPL, bool SOFT, bool VEC, bool SEQ>
__global__ void __launch_bounds__(RT_WARPS * 32, EPL == 8 ? 8 : 10)
    route_bwd_kernel(const RouteBwdArgs a) {
  constexpr int TOKENS = 32 / SEG;
  constexpr uint32_t ALL = SEG == 32 ? FULL : (1u << SEG % 32) - 1;
  __shared__ __align__(16) double sh[RT_WARPS][RT_EMAX];
  behind();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * RT_WARPS + warp) * TOKENS;
  if (t0 >= a.T) return;
  if (a.k > SEG) {  // of SEG = 32 only
    route_bwd_f64<LT>(a, t0, sh[warp]);
    return;
  }
  const int l = lane & (SEG - 1), base = lane - l, e0 = l * EPL;
  const bool real = t0 + lane / SEG < a.T;
  const int64_t t = real ? t0 + lane / SEG : a.T - 1;
  float* dp = reinterpret_cast<float*>(sh[warp]);  // the picks' dp, by slot
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  const bool mine = l < a.k;
  const int e = mine ? a.idx[t * a.k + l] : -1;
  const float wj = mine ? a.w[t * a.k + l] : 0.0f, dwj = mine ? a.dw[t * a.k + l] : 0.0f;
  const bool ok = wj != 0.0f && e >= 0 && e < a.E;
  const int se = ok ? slot<EPL>(base + e / EPL, e % EPL) : 0;
  float x[EPL], sg[EPL];
  load_row(x, row, e0, a.E, VEC, -INFINITY);
  if (SEQ) {
    const uint32_t len = (uint32_t)min(a.seq_len, (int64_t)0x7fffffff);  // T is below 2^31
    load_row(sg, a.seq_grad + (int64_t)((uint32_t)t / len) * a.E, e0, a.E, VEC, 0.0f);
  }
  const float xe = ok ? load1(row + e) : 0.0f;
  // does an expert stand twice among the picks?
  if (ok) dp[se] = __int_as_float(lane);
  __syncwarp();
  const bool twice = __any_sync(FULL, ok && __float_as_int(dp[se]) != lane);
  float g[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) g[q] = 0.0f;
  put(dp, lane, g);
  // affinities, of a softmax times their sum z
  float p[EPL], s1[EPL];  // s1: p (1 - p) of a sigmoid, without the cancellation of 1 - p
  float m = 0.0f;
  if (SOFT) {
    m = x[0];
#pragma unroll
    for (int q = 1; q < EPL; ++q) m = fmaxf(m, x[q]);
    if (SEG == 32) {
      m = warp_max(m);
    } else {
#pragma unroll
      for (int o = 1; o < SEG; o <<= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    }
    if (m == -INFINITY) m = 0.0f;
  }
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    if (SOFT) {
      p[q] = expf(x[q] - m);
    } else {
      const float h = expf(-fabsf(x[q])), r = quick_rcp(1.0f + h);
      p[q] = x[q] >= 0.0f ? r : x[q] < 0.0f ? h * r : x[q];
      s1[q] = h * r * r;
    }
  }
  const float pe = ok ? affinity<SOFT>(xe, m) : 0.0f;
  // all sums in one round: over the picks p, dw w and p dw, over the experts p and p g
  float sum[5] = {pe, ok ? dwj * wj : 0.0f, ok ? pe * dwj : 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    sum[3] += p[q];
    if (SEQ) sum[4] = fmaf(p[q], sg[q], sum[4]);
  }
#pragma unroll
  for (int o = SEG / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 5; ++i) sum[i] += __shfl_xor_sync(FULL, sum[i], o);
  const float z = sum[3], rz = z == 0.0f ? 0.0f : quick_rcp(z);
  // a pick too near the subnormal numbers: its gradient may be an ordinary number
  bool bad = (!SOFT && SEQ && z < RT_SMALL_ALL) || (ok && pe < RT_TINY);
  const bool any = (__ballot_sync(FULL, ok) & ALL << base) != 0;
  const float unit = SOFT ? rz : 1.0f;  // of p
  float d = a.scale * dwj, cp = a.scale * (sum[2] * unit);  // cp: sum of p dp over the picks
  if (a.renorm) {
    bad |= any && sum[0] < RT_SMALL_SUM;
    const float r = any ? 1.0f / sum[0] : 0.0f;  // 1 / sum of the picks' p z
    d = (d - sum[1]) * r * (SOFT ? z : 1.0f);
    cp = a.scale * (sum[2] * r) - (any ? sum[1] : 0.0f);
  }
  bad |= ok && fabsf(d) == INFINITY;  // the factor over a small sum
  if (twice) {  // both terms, in the picks' order
    const unsigned same = __match_any_sync(FULL, ok ? base << 16 | e : -1 - lane);
    float v = 0.0f;
    for (int j = 0; j < 32; ++j) {
      const float o = __shfl_sync(FULL, d, j);
      if (same >> j & 1) v += o;
    }
    d = v;
  }
  __syncwarp();
  if (ok) dp[se] = d;
  __syncwarp();
  get(dp, lane, g);
  const float cg = SEQ ? sum[4] * rz : 0.0f;  // of the affinities that sum to 1
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    if (SOFT) g[q] = p[q] * rz * (SEQ ? g[q] + sg[q] - (cp + cg) : g[q] - cp);
    else g[q] = s1[q] * (SEQ ? g[q] + (sg[q] - cg) * rz : g[q]);
  }
  if (real) store_row(reinterpret_cast<LT*>(a.dlogits) + t * a.E, g, e0, a.E, VEC);
  const uint32_t stopped = __ballot_sync(FULL, bad && real);
  if (stopped)
    for (int i = 0; i < TOKENS; ++i)
      if (stopped >> (i * SEG) & ALL) {
        __syncwarp();  // sh and the row are free
        route_bwd_f64<LT>(a, t0 + i, sh[warp]);
      }
}

// Whether a token takes a few lanes of eight experts each, up to 128 experts: 8 lanes of 64,
// 16 of 128.  With 16384 tokens of 64 experts the forward took 6.8 us instead of 11.3, of
// 128 experts 11.1 instead of 12.9; with 2048 tokens and fewer a warp each is as fast or
// faster (128 experts: 3.2 against 3.7 us), for its shorter chain of steps.  Of 256
// experts, 16 lanes of 16 took 18.3 us instead of 16.5.
bool few_lanes(const moe_dims& dm) {
  return dm.T >= 2560 && dm.E <= 128 && dm.k <= (dm.E <= 64 ? 8 : 16);
}

// Whether rows of E experts from p on can be taken a lane's share at a time: whole pieces
// that start on their alignment.
bool in_pieces(const void* p, int E, int size, bool few = false) {
  const int epl = few ? 8 : E <= 64 ? 2 : E <= 128 ? 4 : 8;
  const int piece = epl * size < 16 ? epl * size : 16;
  return E % epl == 0 && reinterpret_cast<uintptr_t>(p) % piece == 0;
}

// Launches the kernel for a call's settings, as compile-time values.
template <typename F>
void settle(bool v, F f) {
  if (v) f(std::true_type{});
  else f(std::false_type{});
}
template <typename LT, int EPL>
int start(const RouteArgs& a, cudaStream_t st) {
  if constexpr (EPL < 8) {
    constexpr int SEG = EPL * 4, PER = 8;
    if (a.few) {
      const int64_t tokens = RT_WARPS * 32 / SEG, blocks = (a.T + tokens - 1) / tokens;
      int rc = MOE_OK;
      settle(a.softmax, [&](auto soft) {
        settle(a.n_group > 1, [&](auto groups) {
          rc = launch_behind(route_topk_few_kernel<LT, SEG, PER, soft.value, groups.value>, blocks,
                             RT_WARPS * 32, 0, st, a);
        });
      });
      return rc;
    }
  }
  const int64_t blocks = (a.T + RT_WARPS - 1) / RT_WARPS;
  int rc = MOE_OK;
  settle(a.softmax, [&](auto soft) {
    settle(a.vec, [&](auto vec) {
      settle(a.n_group > 1, [&](auto groups) {
        rc = launch_behind(route_topk_kernel<LT, EPL, soft.value, vec.value, groups.value>, blocks,
                           RT_WARPS * 32, 0, st, a);
      });
    });
  });
  return rc;
}
template <typename LT, int SEG, int EPL, bool FEW>
int start_bwd(const RouteBwdArgs& a, cudaStream_t st) {
  const int64_t tokens = RT_WARPS * 32 / SEG, blocks = (a.T + tokens - 1) / tokens;
  int rc = MOE_OK;
  settle(a.softmax, [&](auto soft) {
    settle(FEW || a.vec, [&](auto vec) {
      settle(a.seq_grad != nullptr, [&](auto seq) {
        if constexpr (vec.value || !FEW)
          rc = launch_behind(route_bwd_kernel<LT, SEG, EPL, soft.value, vec.value, seq.value>,
                             blocks, RT_WARPS * 32, 0, st, a);
      });
    });
  });
  return rc;
}
template <typename LT, int EPL>
int start(const RouteBwdArgs& a, cudaStream_t st) {
  if constexpr (EPL < 8)
    if (a.few) return start_bwd<LT, EPL * 4, 8, true>(a, st);
  return start_bwd<LT, 32, EPL, false>(a, st);
}

template <typename LT, typename Args>
int start_for(const Args& a, cudaStream_t st) {
  if (a.E <= 64) return start<LT, 2>(a, st);
  if (a.E <= 128) return start<LT, 4>(a, st);
  return start<LT, 8>(a, st);
}

}  // namespace

int launch_route_topk(const moe_dims& dm, const moe_route_cfg& c, int type, const void* logits,
                      const float* bias, int32_t* idx, float* w, float* probs, void* stream) {
  if (dm.T == 0) return MOE_OK;
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.idx = idx;
  a.w = w;
  a.probs = probs;
  a.T = dm.T;
  a.E = dm.E;
  a.k = dm.k;
  a.n_group = c.topk_group == c.n_group ? 1 : c.n_group;  // all groups kept: no groups
  a.topk_group = c.topk_group;
  a.group_top = c.group_top;
  a.renorm = c.renorm;
  a.softmax = c.score == MOE_SCORE_SOFTMAX;
  a.scale = c.scale;
  a.vec = in_pieces(logits, dm.E, type == MOE_F32 ? 4 : 2) && in_pieces(probs, dm.E, 4) &&
          in_pieces(bias, dm.E, 4);
  a.few = few_lanes(dm) && in_pieces(logits, dm.E, type == MOE_F32 ? 4 : 2, true) &&
          in_pieces(probs, dm.E, 4, true) && in_pieces(bias, dm.E, 4, true);
  if (a.n_group > 1) {  // groups in whole lanes
    const int lanes = dm.E / a.n_group / 8;
    a.few &= lanes * 8 * a.n_group == dm.E && (lanes & (lanes - 1)) == 0;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return type == MOE_F32 ? start_for<float>(a, st) : start_for<__nv_bfloat16>(a, st);
}

int launch_route_bwd(const moe_dims& dm, const moe_route_cfg& c, int type, const void* logits,
                     const int32_t* idx, const float* w, const float* dw, const float* seq_grad,
                     int64_t seq_len, void* dlogits, void* stream) {
  if (dm.T == 0) return MOE_OK;
  RouteBwdArgs a{};
  a.logits = logits;
  a.idx = idx;
  a.w = w;
  a.dw = dw;
  a.seq_grad = seq_grad;
  a.dlogits = dlogits;
  a.T = dm.T;
  a.seq_len = seq_len;
  a.E = dm.E;
  a.k = dm.k;
  a.renorm = c.renorm;
  a.softmax = c.score == MOE_SCORE_SOFTMAX;
  a.scale = c.scale;
  const int size = type == MOE_F32 ? 4 : 2;
  a.vec = in_pieces(logits, dm.E, size) && in_pieces(dlogits, dm.E, size) &&
          in_pieces(seq_grad, dm.E, 4);
  a.few = few_lanes(dm) && in_pieces(logits, dm.E, size, true) &&
          in_pieces(dlogits, dm.E, size, true) && in_pieces(seq_grad, dm.E, 4, true);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return type == MOE_F32 ? start_for<float>(a, st) : start_for<__nv_bfloat16>(a, st);
}

}  // namespace moe
