// grads.cu -- the global norm of many gradient tensors and their clipping.
//
// Passage: dots.llm1 Technical Report, §Training (gradients clipped to a norm).
// HBM-bound: the norm reads every element once, the clipping reads it again and
// writes it once.  The list travels as a kernel argument (up to GL_MAX tensors a
// launch), so nothing is copied to the device and a captured graph holds its own.
//
// A launch splits its tensors into chunks of GL_CHUNK elements of one tensor each;
// CTA b takes chunks b, b + gridDim, ... .  Squares are exact in 64 bits (an FP32
// value's square has 48 significant bits) and are added in 64 bits: no overflow,
// no lost small elements.  Every sum runs in an order fixed by the list's sizes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int GL_MAX = 512;      // tensors per launch
constexpr int GL_CTAS = 592;     // CTAs of a norm launch: one partial sum each
constexpr int GL_THREADS = 256;
constexpr int GL_CHUNK = 16384;  // elements

struct GradEnt {
  const void* data;
  void* out;
  int64_t n;
  int64_t chunk0;  // chunks of the launch's earlier tensors
};

struct GradTable {
  GradEnt e[GL_MAX];
  uint8_t type[GL_MAX];
  int n;
  int64_t chunks;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half* p, float v) { *p = __float2half_rn(v); }

// The tensor that holds a chunk: the last one whose first chunk is not past it.
__device__ __forceinline__ int find(const GradTable& tb, int64_t chunk) {
  int lo = 0, hi = tb.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (tb.e[mid].chunk0 <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ double chunk_sum(const void* data, int64_t i0, int64_t i1) {
  const T* p = reinterpret_cast<const T*>(data);
  double s = 0.0;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
    const double v = to_f32(p[i]);
    s = fma(v, v, s);
  }
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

__global__ void __launch_bounds__(GL_THREADS)
    grad_sumsq_kernel(const __grid_constant__ GradTable tb, double* __restrict__ part) {
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < tb.chunks; c += gridDim.x) {
    const int k = find(tb, c);
    const int64_t i0 = (c - tb.e[k].chunk0) * GL_CHUNK;
    const int64_t i1 = min(i0 + GL_CHUNK, tb.e[k].n);
    if (tb.type[k] == MOE_F32) s += chunk_sum<float>(tb.e[k].data, i0, i1);
    else if (tb.type[k] == MOE_BF16) s += chunk_sum<__nv_bfloat16>(tb.e[k].data, i0, i1);
    else s += chunk_sum<__half>(tb.e[k].data, i0, i1);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(GL_THREADS)
    grad_finish_kernel(const double* __restrict__ part, int64_t n, int accumulate, double* sumsq,
                       float* norm) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) s += part[i];
  s = block_sum(s);
  if (threadIdx.x == 0) {
    if (accumulate) s += *sumsq;
    *sumsq = s;
    if (norm) *norm = (float)sqrt(s);
  }
}

template <typename T>
__device__ void chunk_scale(const void* data, void* out, int64_t i0, int64_t i1, float f) {
  const T* p = reinterpret_cast<const T*>(data);
  T* o = reinterpret_cast<T*>(out);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) from_f32(o + i, to_f32(p[i]) * f);
}

__global__ void __launch_bounds__(GL_THREADS)
    grad_clip_kernel(const __grid_constant__ GradTable tb, const double* __restrict__ sumsq,
                     float max_norm, float* norm, float* coef) {
  const double nm = sqrt(*sumsq);
  const double q = (double)max_norm / (nm + 1e-6);
  const float f = q >= 1.0 ? 1.0f : (float)q;  // a NaN stays one
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (norm) *norm = (float)nm;
    if (coef) *coef = f;
  }
  for (int64_t c = blockIdx.x; c < tb.chunks; c += gridDim.x) {
    const int k = find(tb, c);
    const GradEnt& e = tb.e[k];
    if (f == 1.0f && e.out == e.data) continue;
    const int64_t i0 = (c - e.chunk0) * GL_CHUNK;
    const int64_t i1 = min(i0 + GL_CHUNK, e.n);
    if (tb.type[k] == MOE_F32) chunk_scale<float>(e.data, e.out, i0, i1, f);
    else if (tb.type[k] == MOE_BF16) chunk_scale<__nv_bfloat16>(e.data, e.out, i0, i1, f);
    else chunk_scale<__half>(e.data, e.out, i0, i1, f);
  }
}

// The next launch's table: tensors from *i on, empty ones left out.
void fill(GradTable& tb, const moe_grad* g, int64_t n, int64_t* i) {
  tb.n = 0;
  tb.chunks = 0;
  for (; *i < n && tb.n < GL_MAX; ++*i) {
    const moe_grad& x = g[*i];
    if (x.n == 0) continue;
    GradEnt& e = tb.e[tb.n];
    e.data = x.data;
    e.out = x.out ? x.out : const_cast<void*>(x.data);
    e.n = x.n;
    e.chunk0 = tb.chunks;
    tb.type[tb.n++] = (uint8_t)x.type;
    tb.chunks += (x.n + GL_CHUNK - 1) / GL_CHUNK;
  }
}

int64_t grad_launches(int64_t n) { return n > 0 ? (n + GL_MAX - 1) / GL_MAX : 1; }

}  // namespace

size_t grad_ws_bytes(int64_t n) {
  return align_up((size_t)grad_launches(n) * GL_CTAS * sizeof(double), 256);
}

int launch_grad_norm(const moe_grad* g, int64_t n, int accumulate, double* sumsq, float* norm,
                     void* ws, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(ws);
  int64_t parts = 0;
  for (int64_t i = 0; i < n;) {
    GradTable tb;
    fill(tb, g, n, &i);
    if (tb.n == 0) break;
    const unsigned ctas = (unsigned)(tb.chunks < GL_CTAS ? tb.chunks : GL_CTAS);
    grad_sumsq_kernel<<<ctas, GL_THREADS, 0, st>>>(tb, part + parts);
    parts += ctas;
  }
  grad_finish_kernel<<<1, GL_THREADS, 0, st>>>(part, parts, accumulate, sumsq, norm);
  return cuda_ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
}

int launch_grad_clip(const moe_grad* g, int64_t n, const double* sumsq, float max_norm,
                     float* norm, float* coef, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int64_t i = 0;
  do {
    GradTable tb;
    fill(tb, g, n, &i);
    const int64_t ctas = tb.chunks < GL_CTAS ? (tb.chunks > 0 ? tb.chunks : 1) : GL_CTAS;
    grad_clip_kernel<<<(unsigned)ctas, GL_THREADS, 0, st>>>(tb, sumsq, max_norm, norm, coef);
  } while (i < n);
  return cuda_ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
