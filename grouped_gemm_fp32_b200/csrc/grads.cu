// grads.cu -- the global norm of many gradient tensors and their clipping.
//
// Passage: dots.llm1 Technical Report, §Training (gradients clipped to a norm).
// HBM-bound: the norm reads every element once, the clipping reads it again and
// writes it once.  The list travels as a kernel argument (up to GL_MAX tensors a
// launch), so nothing is copied to the device and a captured graph holds its own.
//
// A launch splits its tensors into chunks of up to GL_CHUNK elements of one tensor each;
// CTA b takes chunks b, b + gridDim, ... .  Squares are exact in 64 bits (an FP32 value's
// square has 48 significant bits) and are added in 64 bits: no overflow, no lost small
// elements.  Every sum runs in an order fixed by the list's sizes and its tensors' addresses
// modulo 16 (whole vectors first).
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int GL_MAX = 512;      // tensors per launch
constexpr int GL_FEW = 48;       // of a launch with the short table
// CTAs of a norm's launch (and its partial sums) and of a clipping's, at most: ten and 24 an
// SM, of which four run at a time.  With four each, 60 M bf16 elements took 67 us instead of
// 62 and 624 M FP32 ones 596 instead of 560: a CTA that is done early makes room.
constexpr int GL_CTAS = 148 * 10;
constexpr int GL_CLIP_CTAS = 148 * 24;
constexpr int GL_THREADS = 256;
constexpr int GL_CHUNK = 32768;  // most elements of a chunk: 16 vectors a thread of bf16
constexpr int GL_CHUNK_MIN = 2048;

struct GradEnt {
  const void* data;
  void* out;
  int64_t n;
  int64_t chunk0;  // chunks of the launch's earlier tensors
};

// N: the most tensors of a launch.  The table is copied at every launch, so a list of few
// tensors goes in a short one.
template <int N>
struct GradTable {
  GradEnt e[N];
  uint8_t type[N];
  int n;
  int chunk;       // elements of a chunk: less than GL_CHUNK where that fills more CTAs
  int64_t chunks;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half* p, float v) { *p = __float2half_rn(v); }

// The tensor that holds a chunk: the last one whose first chunk is not past it.
template <int N>
__device__ __forceinline__ int find(const GradTable<N>& tb, int64_t chunk) {
  int lo = 0, hi = tb.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (tb.e[mid].chunk0 <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The part [v0, v1) of elements [i0, i1) of p that 16-byte vectors cover; the up to 7
// elements on either side are read one by one.
template <typename T>
__device__ __forceinline__ void vector_part(const T* p, int64_t i0, int64_t i1, int64_t& v0,
                                            int64_t& v1) {
  constexpr int N = 16 / sizeof(T);
  const int64_t off = (int64_t)((uintptr_t)p / sizeof(T) % N);  // element of p[0] in its vector
  v0 = min((i0 + off + N - 1) / N * N - off, i1);
  v1 = max((i1 + off) / N * N - off, v0);
}

__device__ __forceinline__ void add_square(double& s, float v) {
  const double d = v;
  s = fma(d, d, s);
}

// The sum of a thread's squares.  FP32 elements are converted; of 16-bit ones a thread has
// twice as many in the same time, so theirs come from the bits: those of |x| as FP32, three
// places down and with 896 added to the exponent, are those of |x| in 64 bits where x is
// normal.  A zero or subnormal x stands there as a number below 2^-126, whose square is
// nothing beside that of a 2^-60.  `top` collects the largest |x|: a run with infinities or
// NaN, or with nothing above 2^-60, is summed again by conversion, and one of zeros is 0.
template <typename T>
struct Squares {
  static constexpr bool BITS = sizeof(T) == 2;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  uint32_t top = 0;  // two 16-bit patterns

  // hi: the pattern of |x| in FP32, three places down; its last 13 bits were zero
  __device__ __forceinline__ static void add_bits(double& to, uint32_t hi) {
    const double d = __hiloint2double((int)(hi + (896u << 20)), 0);
    to = fma(d, d, to);
  }
  __device__ __forceinline__ void add(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (!BITS) {
        add_square(s[i], __uint_as_float(w[i]));
      } else {
        top = __vmaxu2(top, w[i] & 0x7fff7fffu);
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
          add_bits(s[i], (w[i] & 0x7fffu) << 13);
          add_bits(s[i], w[i] >> 3 & 0x0fffe000u);
        } else {  // as FP32 a half is normal or zero
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          const uint32_t a = __float_as_uint(f.x) & 0x7fffffffu;
          const uint32_t b = __float_as_uint(f.y) & 0x7fffffffu;
          add_bits(s[i], a >> 3);
          add_bits(s[i], b >> 3);
        }
      }
    }
  }
  // The run has to be summed by conversion.
  __device__ __forceinline__ bool again() const {
    if constexpr (!BITS) return false;
    constexpr bool BF = std::is_same_v<T, __nv_bfloat16>;
    constexpr uint32_t INF = BF ? 0x7f80u : 0x7c00u, LOW = BF ? (127u - 60u) << 7 : 1u;
    const uint32_t m = max(top >> 16, top & 0xffffu);
    return m >= INF || (m != 0 && m < LOW);
  }
  __device__ __forceinline__ double total() const {
    return BITS && top == 0 ? 0.0 : (s[0] + s[1]) + (s[2] + s[3]);
  }
};

// The squares of elements [i0, i1).
template <typename T>
__device__ __noinline__ double run_sum(const void* data, int64_t i0, int64_t i1) {
  constexpr int N = 16 / sizeof(T), BATCH = 4;
  const T* p = reinterpret_cast<const T*>(data);
  int64_t v0, v1;
  vector_part(p, i0, i1, v0, v1);
  const uint4* v = reinterpret_cast<const uint4*>(p + v0) + threadIdx.x;
  const int64_t n = (v1 - v0) / N - threadIdx.x;  // from this thread's first on
  Squares<T> q;
  auto load = [&](uint4 (&u)[BATCH]) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) u[k] = __ldg(v + k * GL_THREADS);
    v += BATCH * GL_THREADS;
  };
  auto add = [&](const uint4 (&u)[BATCH]) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) q.add(u[k]);
  };
  // two batches take turns, one on its way while the other is added
  int64_t left = n > 0 ? (n - 1) / GL_THREADS + 1 : 0;  // this thread's vectors
  if (left >= BATCH) {
    uint4 a[BATCH], b[BATCH];
    load(a);
    left -= BATCH;
    for (; left >= 2 * BATCH; left -= 2 * BATCH) {
      load(b);
      add(a);
      load(a);
      add(b);
    }
    if (left >= BATCH) {
      load(b);
      left -= BATCH;
      add(a);
      add(b);
    } else {
      add(a);
    }
  }
#pragma unroll 1
  for (; left > 0; --left, v += GL_THREADS) q.add(__ldg(v));
  double s = q.total();
  if (q.again()) {
    s = 0.0;
#pragma unroll 1
    for (int64_t i = threadIdx.x; i < (v1 - v0) / N; i += GL_THREADS)
#pragma unroll 1
      for (int k = 0; k < N; ++k) add_square(s, to_f32(p[v0 + i * N + k]));
  }
  for (int64_t e = i0 + threadIdx.x; e < v0; e += GL_THREADS) add_square(s, to_f32(p[e]));
  for (int64_t e = v1 + threadIdx.x; e < i1; e += GL_THREADS) add_square(s, to_f32(p[e]));
  return s;
}

__device__ double block_sum(double v) {
  __shared__ double sh[GL_THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < GL_THREADS / 32; ++i) v += sh[i];
  return v;
}

template <int N>
__global__ void __launch_bounds__(GL_THREADS, 4)
    grad_sumsq_kernel(const __grid_constant__ GradTable<N> tb, double* __restrict__ part) {
  behind();
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < tb.chunks; c += gridDim.x) {
    const int k = find(tb, c);
    const GradEnt& e = tb.e[k];
    const int64_t i0 = (c - e.chunk0) * tb.chunk, i1 = min(i0 + tb.chunk, e.n);
    if (tb.type[k] == MOE_F32) s += run_sum<float>(e.data, i0, i1);
    else if (tb.type[k] == MOE_BF16) s += run_sum<__nv_bfloat16>(e.data, i0, i1);
    else s += run_sum<__half>(e.data, i0, i1);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm launches' partial sums, the same bits in every CTA that adds them.
__device__ __forceinline__ double sum_parts(const double* part, int64_t n) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += GL_THREADS) s += part[i];
  return block_sum(s);
}

__global__ void __launch_bounds__(GL_THREADS)
    grad_finish_kernel(const double* part, int64_t n, int accumulate, double* sumsq, float* norm) {
  behind();
  double s = sum_parts(part, n);
  if (threadIdx.x == 0) {
    if (accumulate) s += *sumsq;
    *sumsq = s;
    if (norm) *norm = (float)sqrt(s);
  }
}

__device__ __forceinline__ uint4 scale(const uint4& u, float f, const float*) {
  return make_uint4(__float_as_uint(__uint_as_float(u.x) * f),
                    __float_as_uint(__uint_as_float(u.y) * f),
                    __float_as_uint(__uint_as_float(u.z) * f),
                    __float_as_uint(__uint_as_float(u.w) * f));
}
__device__ __forceinline__ uint32_t scale2(uint32_t w, float f, const __nv_bfloat16*) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(__uint_as_float(w << 16) * f,
                                                 __uint_as_float(w & 0xffff0000u) * f);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t scale2(uint32_t w, float f, const __half*) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
  const __half2 r = __floats2half2_rn(v.x * f, v.y * f);
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint4 scale(const uint4& u, float f, const T* t) {
  return make_uint4(scale2(u.x, f, t), scale2(u.y, f, t), scale2(u.z, f, t), scale2(u.w, f, t));
}

// 16 bytes from byte 4 WS + bits / 8 of the 32 bytes a, b on.
template <int WS>
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, uint32_t bits) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return make_uint4(__funnelshift_r(w[WS], w[WS + 1], bits),
                    __funnelshift_r(w[WS + 1], w[WS + 2], bits),
                    __funnelshift_r(w[WS + 2], w[WS + 3], bits),
                    __funnelshift_r(w[WS + 3], w[WS + 4], bits));
}

// Vectors of out that are 16-byte aligned, out of data that may not be: `u` points at the
// 16 bytes that hold the first one's first element, which stands 4 WS + bits / 8 bytes in.
// WS < 0: data is aligned too.  A warp takes neighbouring vectors, some a lane at a time; the words
// that a vector needs of the next one come from the next lane.
template <typename T, int WS>
__device__ __noinline__ void scale_vectors(const uint4* u, uint4* o, int n, uint32_t bits,
                                           float f) {
  constexpr int BATCH = WS < 0 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  int i = (threadIdx.x >> 5) * 32 * BATCH;
  for (; i + 32 * BATCH <= n; i += GL_THREADS * BATCH) {
    uint4 a[BATCH + 1];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) a[k] = u[i + 32 * k + lane];
    if constexpr (WS >= 0) a[BATCH] = lane == 0 ? u[i + 32 * BATCH] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if constexpr (WS >= 0) {
        // lane 31's next vector is lane 0's of the next 32
        const uint4 g = lane == 0 ? a[k + 1] : a[k];
        const int from = lane + 1 & 31;
        uint4 b = make_uint4(0, 0, 0, 0);
        b.x = __shfl_sync(0xffffffffu, g.x, from);
        if (WS > 0) b.y = __shfl_sync(0xffffffffu, g.y, from);
        if (WS > 1) b.z = __shfl_sync(0xffffffffu, g.z, from);
        if (WS > 2) b.w = __shfl_sync(0xffffffffu, g.w, from);
        o[i + 32 * k + lane] = scale(shifted<WS>(a[k], b, bits), f, (const T*)nullptr);
      } else {
        o[i + 32 * k + lane] = scale(a[k], f, (const T*)nullptr);
      }
    }
  }
  // fewer than a warp's share are left
  i = n / (32 * BATCH) * (32 * BATCH) + threadIdx.x;
  if (i < n) {
    uint4 a = u[i];
    if constexpr (WS >= 0) a = shifted<WS>(a, u[i + 1], bits);
    o[i] = scale(a, f, (const T*)nullptr);
  }
}

// out[i] = f data[i] for a chunk [i0, i1) of a tensor of n elements.
template <typename T>
__device__ void chunk_scale(const void* data, void* out, int64_t i0, int64_t i1, int64_t n,
                            float f) {
  constexpr int N = 16 / sizeof(T);
  const T* p = reinterpret_cast<const T*>(data);
  T* o = reinterpret_cast<T*>(out);
  int64_t v0, v1;
  vector_part(o, i0, i1, v0, v1);
  // where data[v0] stands in its 16 bytes; the 16-byte pieces read must lie in the tensor
  const int in = (int)((uintptr_t)(p + v0) % 16 / sizeof(T));
  if (in != 0 && v1 > v0) {
    if (v0 < in) v0 += N;
    while (v1 > v0 && v1 + N - in > n) v1 -= N;
  }
  if (v1 > v0) {
    const uint4* u = reinterpret_cast<const uint4*>(p + v0 - in);
    uint4* w = reinterpret_cast<uint4*>(o + v0);
    const int nv = (int)((v1 - v0) / N);
    const uint32_t byte = in * sizeof(T), bits = byte % 4 * 8;
    if (byte == 0) scale_vectors<T, -1>(u, w, nv, 0, f);
    else if (byte < 4) scale_vectors<T, 0>(u, w, nv, bits, f);
    else if (byte < 8) scale_vectors<T, 1>(u, w, nv, bits, f);
    else if (byte < 12) scale_vectors<T, 2>(u, w, nv, bits, f);
    else scale_vectors<T, 3>(u, w, nv, bits, f);
  } else {
    v0 = v1 = i1;
  }
  for (int64_t i = i0 + threadIdx.x; i < v0; i += GL_THREADS) from_f32(o + i, to_f32(p[i]) * f);
  for (int64_t i = v1 + threadIdx.x; i < i1; i += GL_THREADS) from_f32(o + i, to_f32(p[i]) * f);
}

// All chunks with a factor below FP32's normal range, which would lose its bits there.
template <typename T>
__device__ void chunk_scale_f64(const void* data, void* out, int64_t i0, int64_t i1,
                                             double f) {
  const T* p = reinterpret_cast<const T*>(data);
  T* o = reinterpret_cast<T*>(out);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += GL_THREADS)
    from_f32(o + i, (float)(to_f32(p[i]) * f));
}

template <int N>
__device__ __noinline__ void scale_f64(const GradTable<N>& tb, double f) {
  for (int64_t c = blockIdx.x; c < tb.chunks; c += gridDim.x) {
    const int k = find(tb, c);
    const GradEnt& e = tb.e[k];
    const int64_t i0 = (c - e.chunk0) * tb.chunk, i1 = min(i0 + tb.chunk, e.n);
    if (tb.type[k] == MOE_F32) chunk_scale_f64<float>(e.data, e.out, i0, i1, f);
    else if (tb.type[k] == MOE_BF16) chunk_scale_f64<__nv_bfloat16>(e.data, e.out, i0, i1, f);
    else chunk_scale_f64<__half>(e.data, e.out, i0, i1, f);
  }
}

// parts > 0: the sum of squares is that of the norm launches' partial sums, which every
// CTA adds up for itself, and is written to sumsq; otherwise sumsq is given.  The chunks
// are taken in the reverse of the norm's order: what it read last may still be in the L2.
template <int N>
__global__ void __launch_bounds__(GL_THREADS, 4)
    grad_clip_kernel(const __grid_constant__ GradTable<N> tb, const double* part, int64_t parts,
                     double* sumsq, float max_norm, float* norm, float* coef) {
  behind();
  const double ss = parts > 0 ? sum_parts(part, parts) : *sumsq;
  const double nm = sqrt(ss);
  // no limit: no clipping, whatever the norm
  const double q = max_norm == INFINITY ? 1.0 : (double)max_norm / (nm + 1e-6);
  const float f = q >= 1.0 ? 1.0f : (float)q;  // a NaN stays one
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (parts > 0) *sumsq = ss;
    if (norm) *norm = (float)nm;
    if (coef) *coef = f;
  }
  if (q < 0x1p-126 && q > 0.0) {
    scale_f64(tb, q);
    return;
  }
  for (int64_t r = blockIdx.x; r < tb.chunks; r += gridDim.x) {
    const int64_t c = tb.chunks - 1 - r;
    const int k = find(tb, c);
    const GradEnt& e = tb.e[k];
    if (f == 1.0f && e.out == e.data) continue;
    const int64_t i0 = (c - e.chunk0) * tb.chunk;
    const int64_t i1 = min(i0 + tb.chunk, e.n);
    if (tb.type[k] == MOE_F32) chunk_scale<float>(e.data, e.out, i0, i1, e.n, f);
    else if (tb.type[k] == MOE_BF16) chunk_scale<__nv_bfloat16>(e.data, e.out, i0, i1, e.n, f);
    else chunk_scale<__half>(e.data, e.out, i0, i1, e.n, f);
  }
}

// The next launch's table: tensors from *i on, empty ones left out.
template <int N>
void fill(GradTable<N>& tb, const moe_grad* g, int64_t n, int64_t* i) {
  tb.n = 0;
  int64_t total = 0;
  for (; *i < n && tb.n < N; ++*i) {
    const moe_grad& x = g[*i];
    if (x.n == 0) continue;
    GradEnt& e = tb.e[tb.n];
    e.data = x.data;
    e.out = x.out ? x.out : const_cast<void*>(x.data);
    e.n = x.n;
    total += x.n;
    tb.type[tb.n++] = (uint8_t)x.type;
  }
  tb.chunk = GL_CHUNK;
  while (tb.chunk > GL_CHUNK_MIN && total / tb.chunk < GL_CTAS) tb.chunk /= 2;
  tb.chunks = 0;
  for (int k = 0; k < tb.n; ++k) {
    tb.e[k].chunk0 = tb.chunks;
    tb.chunks += (tb.e[k].n + tb.chunk - 1) / tb.chunk;
  }
}

int64_t grad_launches(int64_t n) { return n > 0 ? (n + GL_MAX - 1) / GL_MAX : 1; }

}  // namespace

size_t grad_ws_bytes(int64_t n) {
  return align_up((size_t)grad_launches(n) * GL_CTAS * sizeof(double), 256);
}

// The norm's launches over a list; returns how many partial sums they leave in part.
template <int N>
static int sumsq_with(const moe_grad* g, int64_t n, double* part, int64_t* parts,
                      cudaStream_t st) {
  *parts = 0;
  for (int64_t i = 0; i < n;) {
    GradTable<N> tb;
    fill(tb, g, n, &i);
    if (tb.n == 0) break;
    const int64_t ctas = tb.chunks < GL_CTAS ? tb.chunks : GL_CTAS;
    const int rc = launch_behind(grad_sumsq_kernel<N>, ctas, GL_THREADS, 0, st, tb, part + *parts);
    if (rc != MOE_OK) return rc;
    *parts += ctas;
  }
  return MOE_OK;
}
static int sumsq_launches(const moe_grad* g, int64_t n, double* part, int64_t* parts,
                          cudaStream_t st) {
  return n <= GL_FEW ? sumsq_with<GL_FEW>(g, n, part, parts, st)
                     : sumsq_with<GL_MAX>(g, n, part, parts, st);
}

int launch_grad_norm(const moe_grad* g, int64_t n, int accumulate, double* sumsq, float* norm,
                     void* ws, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(ws);
  int64_t parts;
  const int rc = sumsq_launches(g, n, part, &parts, st);
  if (rc != MOE_OK) return rc;
  return launch_behind(grad_finish_kernel, 1, GL_THREADS, 0, st, part, parts, accumulate, sumsq,
                       norm);
}

// The clipping's launches, in the list's order (each takes its own chunks from the last one
// on).  parts > 0: after the norm's, by its partial sums.
template <int N>
static int clip_with(const moe_grad* g, int64_t n, const double* part, int64_t parts,
                     double* sumsq, float max_norm, float* norm, float* coef, cudaStream_t st) {
  int64_t i = 0;
  do {
    GradTable<N> tb;
    fill(tb, g, n, &i);
    const int64_t ctas = tb.chunks < GL_CLIP_CTAS ? (tb.chunks > 0 ? tb.chunks : 1) : GL_CLIP_CTAS;
    const int rc = launch_behind(grad_clip_kernel<N>, ctas, GL_THREADS, 0, st, tb, part, parts,
                                 sumsq, max_norm, norm, coef);
    if (rc != MOE_OK) return rc;
  } while (i < n);
  return MOE_OK;
}
static int clip_launches(const moe_grad* g, int64_t n, const double* part, int64_t parts,
                         double* sumsq, float max_norm, float* norm, float* coef,
                         cudaStream_t st) {
  return n <= GL_FEW ? clip_with<GL_FEW>(g, n, part, parts, sumsq, max_norm, norm, coef, st)
                     : clip_with<GL_MAX>(g, n, part, parts, sumsq, max_norm, norm, coef, st);
}

int launch_grad_clip(const moe_grad* g, int64_t n, const double* sumsq, float max_norm,
                     float* norm, float* coef, void* stream) {
  return clip_launches(g, n, nullptr, 0, const_cast<double*>(sumsq), max_norm, norm, coef,
                       reinterpret_cast<cudaStream_t>(stream));
}

int launch_grad_clip_norm(const moe_grad* g, int64_t n, float max_norm, double* sumsq,
                          float* norm, float* coef, void* ws, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(ws);
  int64_t parts;
  const int rc = sumsq_launches(g, n, part, &parts, st);
  if (rc != MOE_OK) return rc;
  if (parts == 0 && !cuda_ok(cudaMemsetAsync(sumsq, 0, sizeof(double), st))) return MOE_ERR_CUDA;
  return clip_launches(g, n, part, parts, sumsq, max_norm, norm, coef, st);
}

}  // namespace moe
