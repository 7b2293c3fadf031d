// route.cu -- the router's choice from given logits, and its backward.
//
// Passage: dots.llm1 Technical Report, §Architecture "Mixture of Experts layer"
// and "Load balancing" (top-k of the affinities; the bias only decides the
// choice).  Sigmoid affinities, expert groups and a factor on the weights have no
// counterpart on the pages; the formulas stand in include/moe.h.
//
// One warp per token, lane l holding the EPL consecutive experts from l EPL on.
//
// The choice has to be the one of 64-bit arithmetic, at the price of 32 bits: scores are
// computed in FP32 with a bound on their error (margins below), and the order found stands
// where neighbouring scores differ by more than the bound, or by nothing in 64 bits
// either (equal logits and biases).  Where the check fails, about one token in a thousand,
// the few experts in question are ordered by their scores in 64 bits (refine), and so are
// groups (refine_groups); only tokens beyond FP32's range are done in 64 bits whole.  What bounds the calls is instruction issue (about
// 250 a token for 128 experts), so a pick costs one reduction, a ballot and a few selects:
// each lane keeps its two best scores, and which expert a pick was is looked up once, by
// lane j for pick j.
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
    union {
      double s64[RT_EMAX];  // scores by expert, then group scores
      struct {
        float s[RT_EMAX], score[RT_EMAX];
      };
    };
    int keep[RT_EMAX];
  } group;
};

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
      of_group[g] = a.group_top == 2 ? b1 + b2 : b1;
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

template <bool SOFT>
__device__ __forceinline__ float affinity(float x, float m) {
  return SOFT ? expf(x - m) : quick_rcp(1.0f + expf(-x));
}

// A lane's best values, descending: all of them, or four of eight.
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
      if constexpr (EPL == 8) {  // the larger half of two descending fours, then in order
        sort4(a + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) a[q] = max(a[q], a[7 - q]);
        order(a[0], a[2]);
        order(a[1], a[3]);
        order(a[0], a[1]);
        order(a[2], a[3]);
      }
    }
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = a[q];
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
    score[i] = a.group_top == 2 ? b1 + b2 : b1;
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

// Gives the experts of groups that are not kept the score -inf.  two_dp: twice an
// affinity's error; m: the largest logit, for refine_groups.
template <typename LT, int EPL>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, const LT* row, float m,
                                            RouteShared& sh, float (&s)[EPL], float two_dp) {
  const int lane = threadIdx.x & 31, e0 = lane * EPL;
  const int size = a.E / a.n_group, lanes = size / EPL;
  // of the groups that this lane compares, ordered: the lowest score kept, less its error,
  // and the highest that is not, and its error.  An affinity's error and a rounding for each
  // of a score's terms, and its own
  uint32_t low = 0xffffffffu, high = 0;
  float err = 0.0f;
  auto score = [&](float b1, float b2) {
    const float t = a.group_top == 2 ? fabsf(b1) + fabsf(b2) : fabsf(b1);
    err = two_dp + (t < INFINITY ? 0x1p-22f * t : 0.0f);
    return a.group_top == 2 ? b1 + b2 : b1;
  };
  auto clear = [&]() {
    const float lo = unordered(__reduce_min_sync(FULL, low));
    const uint32_t most = __reduce_max_sync(FULL, high);
    return lo > unordered(most) || most <= ORD_NEG_INF;
  };
  auto sort_out = [&](float mine, bool keep) {
    if (keep) low = min(low, ordered(mine - err));
    else high = max(high, ordered(mine + err));
    if (mine != mine) high = 0xffffffffu;  // inf - inf
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

// The picks' order in 64 bits where FP32 does not settle it: of the experts whose keys are
// `least` or more, the first picks of the token, one a lane (ascending).  `e`: lane j's pick.
// False where there are more than 32.
template <typename LT, int EPL>
__device__ __noinline__ bool refine(const RouteArgs& a, const LT* row, float m, uint32_t least,
                                    RouteShared& sh, int& e) {
  const int lane = threadIdx.x & 31, e0 = lane * EPL;
  int mine = 0;
#pragma unroll 1
  for (int q = 0; q < EPL; ++q) mine += sh.f32.key[slot<EPL>(lane, q)] >= least;
  int at = mine;  // those up to this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL, at, o);
    if (lane >= o) at += v;
  }
  const int n = __shfl_sync(FULL, at, 31);
  if (n > 32) return false;
  at -= mine;
  uint32_t bits = 0;
#pragma unroll 1
  for (int q = 0; q < EPL; ++q) bits |= (sh.f32.key[slot<EPL>(lane, q)] >= least ? 1u : 0u) << q;
  __syncwarp();
  for (; bits; bits &= bits - 1) sh.f32.key[at++] = e0 + __ffs(bits) - 1;
  __syncwarp();
  const int c = lane < n ? (int)sh.f32.key[lane] : 0;
  double x = load1(row + c), rz = 1.0;
  if (a.softmax) {
    double z = 0.0;
#pragma unroll 1
    for (int q = 0; q < EPL; ++q)
      if (e0 + q < a.E) z += exp((double)load1(row + e0 + q) - (double)m);
    rz = 1.0 / warp_sum(z);
    x = exp(x - (double)m) * rz;
  } else {
    x = 1.0 / (1.0 + exp(-x));
  }
  x += (double)a.bias[c];
  int rank = 0;
  for (int h = 0; h < n; ++h) {
    const double v = __shfl_sync(FULL, x, h);
    rank += v > x || (v == x && h < lane);
  }
  __syncwarp();
  if (lane < n) sh.f32.key[rank] = c;
  __syncwarp();
  if (lane < n && lane < a.k) e = (int)sh.f32.key[lane];
  return true;
}

// A token in 32 bits; false where that does not settle the choice or the weights.
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
__device__ __forceinline__ bool route_token(const RouteArgs& a, int64_t t, RouteShared& sh) {
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
  if (!(z > RT_SMALL_ALL)) return false;  // nearly nothing, nothing, or a NaN
  const float rz = quick_rcp(z);
  float s[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) s[q] = p[q] * rz;
  if (a.probs) store_row(a.probs + t * a.E, s, e0, a.E, VEC);
  const float two_dp = SOFT ? 0x1p-18f * rz : 0x1p-21f;
  // scores; without a bias the logits rank the experts, exactly
  if (bias || GROUPS) {
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      if (!SOFT) s[q] = p[q];
      if (bias) s[q] = fmaxf(s[q] + b[q], -INFINITY);  // a NaN ranks as -inf
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
      if (__any_sync(FULL, gone == Best<EPL>::N)) {
        // a lane is out of its best: the ones below the last
        if (gone == Best<EPL>::N) {
          int same = Best<EPL>::N;  // picks equal to the last
#pragma unroll
          for (int q = 0; q < EPL; ++q) same -= u[q] > last;
#pragma unroll
          for (int q = 0; q < EPL; ++q)
            if (u[q] > last || (u[q] == last && same-- > 0)) u[q] = 0;
          best.of(u);
          gone = 0;
        }
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
  int e = mine ? src * EPL + __ffs(where) - 1 : 0;
  if (bias) {
    const uint32_t down = __shfl_down_sync(FULL, key, 1);
    const float sc = unordered(key), dn = unordered(down);
    bool near = lane + 1 < a.k && down != ORD_NEG_INF &&
                !(sc - dn > two_dp + 0x1p-23f * (fabsf(sc) + fabsf(dn)));
    if (__any_sync(FULL, near)) {  // equal in 64 bits too?
      const int en = __shfl_down_sync(FULL, e, 1);
      near = near && !(load1(row + e) == load1(row + en) && a.bias[e] == a.bias[en]);
    }
    // and the first that is not picked
    const uint32_t after = __reduce_max_sync(FULL, best.v[0]);
    const float sl = unordered(last), margin = two_dp + 0x1p-22f * fabsf(sl);
    const uint32_t least = last == ORD_NEG_INF ? last + 1 : ordered(sl - margin);
    if (after > ORD_NEG_INF && after >= least) {  // equal in 64 bits too?
      const int el = __shfl_sync(FULL, e, a.k - 1);
      const float xl = load1(row + el), bl = a.bias[el];
      get(sh.f32.key, lane, u);
#pragma unroll
      for (int q = 0; q < EPL; ++q)
        if (u[q] >= least && u[q] <= last)
          near |= !(u[q] == last && load1(row + e0 + q) == xl && a.bias[e0 + q] == bl);
    }
    if (__any_sync(FULL, near) && !refine<LT, EPL>(a, row, m, least, sh, e)) return false;
  }
  // not: nothing was left to choose from (the last picks only, whatever order the others have)
  const bool some = mine && key != ORD_NEG_INF;
  const float pe = some ? sh.f32.p[slot<EPL>(e / EPL, e % EPL)] : 0.0f;
  const float sum = warp_sum(pe);
  bool bad = some && !(sum > RT_SMALL_SUM);
  if (some && pe < RT_TINY) bad |= load1(row + e) - m > -140.0f;
  if (__any_sync(FULL, bad)) return false;
  if (mine) {
    const float f = a.renorm ? (sum == 0.0f ? 0.0f : a.scale * quick_rcp(sum)) : a.scale * (SOFT ? rz : 1.0f);
    a.idx[t * a.k + lane] = e;
    a.w[t * a.k + lane] = pe * f;
  }
  return true;
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
  if (a.k > 32 || !route_token<LT, EPL, SOFT, VEC, GROUPS>(a, t, sh[warp]))
    route_token_f64<LT>(a, t, sh[warp]);
}

struct RouteBwdArgs {
  const void* logits;
  const int32_t* idx;
  const float *w, *dw, *seq_grad;
  void* dlogits;
  int64_t T, seq_len;
  int E, k, renorm, softmax;
  int vec;  // as in RouteArgs, of logits, seq_grad and dlogits
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

// A token with at most 32 picks, lane j looking after pick j; false where its affinities
// leave FP32's range.  sh: [2][RT_EMAX], by slot.  What bounds it is latency, so the sums
// run side by side: a softmax's sum of p dp over the picks comes from that of p dw.
template <typename LT, int EPL, bool SOFT, bool VEC, bool SEQ>
__device__ __forceinline__ bool route_bwd_token(const RouteBwdArgs& a, int64_t t, float* sh) {
  const int lane = threadIdx.x & 31, e0 = lane * EPL;
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  const bool mine = lane < a.k;
  const int e = mine ? a.idx[t * a.k + lane] : -1;
  const float wj = mine ? a.w[t * a.k + lane] : 0.0f, dwj = mine ? a.dw[t * a.k + lane] : 0.0f;
  const bool ok = wj != 0.0f && e >= 0 && e < a.E;
  const int se = ok ? slot<EPL>(e / EPL, e % EPL) : 0;
  float* ps = sh;            // affinities
  float* dp = sh + RT_EMAX;  // the picks' dp
  float x[EPL], sg[EPL];
  load_row(x, row, e0, a.E, VEC, -INFINITY);
  if (SEQ) {
    const uint32_t len = (uint32_t)min(a.seq_len, (int64_t)0x7fffffff);  // T is below 2^31
    load_row(sg, a.seq_grad + (int64_t)((uint32_t)t / len) * a.E, e0, a.E, VEC, 0.0f);
  }
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
    m = warp_max(m);
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
  put(ps, lane, p);
  __syncwarp();
  const float pe = ok ? ps[se] : 0.0f;
  // all sums in one round: over the picks p, dw w and p dw, over the experts p and p g
  float sum[5] = {pe, ok ? dwj * wj : 0.0f, ok ? pe * dwj : 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    sum[3] += p[q];
    if (SEQ) sum[4] = fmaf(p[q], sg[q], sum[4]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < 5; ++i) sum[i] += __shfl_xor_sync(FULL, sum[i], o);
  const float z = sum[3], rz = z == 0.0f ? 0.0f : quick_rcp(z);
  if (!SOFT && SEQ && z < RT_SMALL_ALL) return false;
  const bool any = __any_sync(FULL, ok);
  const float unit = SOFT ? rz : 1.0f;  // of p
  float d = a.scale * dwj, cp = a.scale * sum[2] * unit;  // cp: sum of p dp over the picks
  if (a.renorm) {
    if (any && sum[0] < RT_SMALL_SUM) return false;
    const float r = any ? 1.0f / sum[0] : 0.0f;  // 1 / sum of the picks' p z
    d = (d - sum[1]) * r * (SOFT ? z : 1.0f);
    cp = a.scale * sum[2] * r - (any ? sum[1] : 0.0f);
  }
  if (twice) {  // both terms, in the picks' order
    const unsigned same = __match_any_sync(FULL, ok ? e : -1 - lane);
    float v = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const float o = __shfl_sync(FULL, d, j);
      if (same >> j & 1) v += o;
    }
    d = v;
  }
  if (ok) dp[se] = d;
  __syncwarp();
  get(dp, lane, g);
  const float cg = SEQ ? sum[4] * rz : 0.0f;  // of the affinities that sum to 1
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    if (SOFT) g[q] = p[q] * rz * (SEQ ? g[q] + sg[q] - (cp + cg) : g[q] - cp);
    else g[q] = s1[q] * (SEQ ? g[q] + (sg[q] - cg) * rz : g[q]);
  }
  store_row(reinterpret_cast<LT*>(a.dlogits) + t * a.E, g, e0, a.E, VEC);
  return true;
}

template <typename LT, int EPL, bool SOFT, bool VEC, bool SEQ>
__global__ void __launch_bounds__(RT_WARPS * 32, EPL == 8 ? 8 : 10)
    route_bwd_kernel(const RouteBwdArgs a) {
  __shared__ __align__(16) double sh[RT_WARPS][RT_EMAX];
  behind();
  const int warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp;
  if (t >= a.T) return;
  float* f32 = reinterpret_cast<float*>(sh[warp]);
  if (a.k > 32 || !route_bwd_token<LT, EPL, SOFT, VEC, SEQ>(a, t, f32))
    route_bwd_f64<LT>(a, t, sh[warp]);
}

// Whether rows of E experts from p on can be taken EPL at a time: whole pieces that start
// on their alignment.
bool in_pieces(const void* p, int E, int size) {
  const int epl = E <= 64 ? 2 : E <= 128 ? 4 : 8;
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
template <typename LT, int EPL>
int start(const RouteBwdArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.T + RT_WARPS - 1) / RT_WARPS;
  int rc = MOE_OK;
  settle(a.softmax, [&](auto soft) {
    settle(a.vec, [&](auto vec) {
      settle(a.seq_grad != nullptr, [&](auto seq) {
        rc = launch_behind(route_bwd_kernel<LT, EPL, soft.value, vec.value, seq.value>, blocks,
                           RT_WARPS * 32, 0, st, a);
      });
    });
  });
  return rc;
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return type == MOE_F32 ? start_for<float>(a, st) : start_for<__nv_bfloat16>(a, st);
}

}  // namespace moe
