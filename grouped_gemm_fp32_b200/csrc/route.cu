// route.cu -- the router's choice from given logits, and its backward.
//
// Passage: dots.llm1 Technical Report, §Architecture "Mixture of Experts layer"
// and "Load balancing" (top-k of the affinities; the bias only decides the
// choice).  Sigmoid affinities, expert groups and a factor on the weights have no
// counterpart on the pages; the formulas stand in include/moe.h.
//
// One warp per token, lane l holding the EPL consecutive experts from l EPL on.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int RT_WARPS = 4;
constexpr unsigned FULL = 0xffffffffu;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  float* probs;
  int64_t T;
  int E, k, n_group, topk_group, group_top, renorm, softmax;
  float scale;
};

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename LT, int EPL>
__global__ void __launch_bounds__(RT_WARPS * 32) route_topk_kernel(const RouteArgs a) {
  __shared__ double s_sh[RT_WARPS][256];  // scores, then the picks' affinities
  __shared__ double g_sh[RT_WARPS][256];  // group scores
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp;
  if (t >= a.T) return;
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  const int e0 = lane * EPL;
  float x[EPL];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    x[q] = e0 + q < a.E ? load1(row + e0 + q) : -INFINITY;
    m = fmaxf(m, x[q]);
  }
  m = warp_max(m);
  // affinities; a logit of -inf takes its expert out, also where all are -inf
  double p[EPL], z = 0.0;
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    if (x[q] == -INFINITY) p[q] = 0.0;
    else if (a.softmax) p[q] = exp((double)x[q] - (double)m);
    else p[q] = 1.0 / (1.0 + exp(-(double)x[q]));
    z += p[q];
  }
  z = warp_sum(z);
  const double rz = z == 0.0 ? 0.0 : 1.0 / z;
  double key[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    const int e = e0 + q;
    const double prob = p[q] * rz;
    if (e < a.E && a.probs) a.probs[t * a.E + e] = (float)prob;
    if (a.softmax) p[q] = prob;
    key[q] = a.bias == nullptr ? p[q] : e < a.E ? p[q] + (double)a.bias[e] : 0.0;
    if (x[q] == -INFINITY || key[q] != key[q]) key[q] = -INFINITY;
    if (e < a.E) s_sh[warp][e] = key[q];
  }
  __syncwarp();
  uint32_t out = 0;  // experts (a bit per q) of groups that are not kept
  if (a.n_group > 1) {
    const int size = a.E / a.n_group;
    for (int g = lane; g < a.n_group; g += 32) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const double v = s_sh[warp][g * size + i];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      g_sh[warp][g] = a.group_top == 2 ? b1 + b2 : b1;
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      const int e = e0 + q;
      if (e >= a.E) continue;
      const int g = e / size;
      const double mine = g_sh[warp][g];
      int before = 0;
      for (int h = 0; h < a.n_group; ++h) {
        const double v = g_sh[warp][h];
        before += v > mine || (v == mine && h < g);
      }
      if (before >= a.topk_group) out |= 1u << q;
    }
  }
  __syncwarp();
  uint32_t alive = 0;
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    // without a bias the logits rank the experts: the same order, and no rounding in it
    if (a.bias == nullptr && key[q] != -INFINITY) key[q] = x[q];
    if (a.bias == nullptr && x[q] != x[q]) key[q] = -INFINITY;
    if (out >> q & 1) key[q] = -INFINITY;
    if (e0 + q < a.E) alive |= 1u << q;
  }
  double sum = 0.0;
  for (int j = 0; j < a.k; ++j) {
    double bk = -INFINITY, bp = 0.0;
    int be = 0x7fffffff;
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if ((alive >> q & 1) && (be == 0x7fffffff || key[q] > bk)) {
        bk = key[q];
        be = e0 + q;
        bp = p[q];
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ok = __shfl_xor_sync(FULL, bk, o), op = __shfl_xor_sync(FULL, bp, o);
      const int oe = __shfl_xor_sync(FULL, be, o);
      if (oe != 0x7fffffff && (be == 0x7fffffff || ok > bk || (ok == bk && oe < be))) {
        bk = ok;
        be = oe;
        bp = op;
      }
    }
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if (e0 + q == be) alive &= ~(1u << q);
    if (bk == -INFINITY && bp == bp) bp = 0.0;  // nothing was left to choose from
    sum += bp;
    if (lane == 0) {
      a.idx[t * a.k + j] = be;
      s_sh[warp][j] = bp;
    }
  }
  __syncwarp();
  const double f = a.renorm ? (sum == 0.0 ? 0.0 : a.scale / sum) : (double)a.scale;
  for (int j = lane; j < a.k; j += 32) a.w[t * a.k + j] = (float)(s_sh[warp][j] * f);
}

struct RouteBwdArgs {
  const void* logits;
  const int32_t* idx;
  const float *w, *dw, *seq_grad;
  void* dlogits;
  int64_t T, seq_len;
  int E, k, renorm, softmax;
  float scale;
};

template <typename LT, int EPL>
__global__ void __launch_bounds__(RT_WARPS * 32) route_bwd_kernel(const RouteBwdArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp;
  if (t >= a.T) return;
  const LT* row = reinterpret_cast<const LT*>(a.logits) + t * a.E;
  const int e0 = lane * EPL;
  float x[EPL], p[EPL], dp[EPL];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    x[q] = e0 + q < a.E ? load1(row + e0 + q) : -INFINITY;
    m = fmaxf(m, x[q]);
    dp[q] = 0.0f;
  }
  m = warp_max(m);
  float z = 0.0f;
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    if (x[q] == -INFINITY) p[q] = 0.0f;
    else if (a.softmax) p[q] = expf(x[q] - m);
    else p[q] = 1.0f / (1.0f + expf(-x[q]));
    z += p[q];
  }
  z = warp_sum(z);
  const float rz = z == 0.0f ? 0.0f : 1.0f / z;
  if (a.softmax) {
#pragma unroll
    for (int q = 0; q < EPL; ++q) p[q] *= rz;
  }
  // the picks: their affinities' sum and the gradients' product with the weights
  float zc = 0.0f, dot = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int e = a.idx[t * a.k + j];
    const float wj = a.w[t * a.k + j];
    if (wj == 0.0f || e < 0 || e >= a.E) continue;
    dot += a.dw[t * a.k + j] * wj;
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if (e0 + q == e) zc += p[q];
  }
  zc = warp_sum(zc);
  const float rzc = a.renorm ? 1.0f / zc : 1.0f;
  if (!a.renorm) dot = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int e = a.idx[t * a.k + j];
    const float wj = a.w[t * a.k + j];
    if (wj == 0.0f || e < 0 || e >= a.E) continue;
    const float d = (a.scale * a.dw[t * a.k + j] - dot) * rzc;
#pragma unroll
    for (int q = 0; q < EPL; ++q)
      if (e0 + q == e) dp[q] += d;
  }
  if (a.seq_grad != nullptr) {
    const float* g = a.seq_grad + (t / a.seq_len) * a.E;
    float ge[EPL], c = 0.0f;
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      ge[q] = e0 + q < a.E ? g[e0 + q] : 0.0f;
      if (!a.softmax) c += p[q] * rz * ge[q];
    }
    if (!a.softmax) c = warp_sum(c);
#pragma unroll
    for (int q = 0; q < EPL; ++q) dp[q] += a.softmax ? ge[q] : (ge[q] - c) * rz;
  }
  float c = 0.0f;
  if (a.softmax) {
#pragma unroll
    for (int q = 0; q < EPL; ++q) c += p[q] * dp[q];
    c = warp_sum(c);
  }
  LT* out = reinterpret_cast<LT*>(a.dlogits) + t * a.E;
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    if (e0 + q >= a.E) continue;
    float v;
    if (a.softmax) {
      v = p[q] * (dp[q] - c);
    } else {  // p (1 - p) without the cancellation of 1 - p
      const float e = expf(-fabsf(x[q]));
      v = dp[q] * (e / ((1.0f + e) * (1.0f + e)));
    }
    store1(out + e0 + q, v);
  }
}

template <typename LT>
int route_topk(const RouteArgs& a, cudaStream_t st) {
  const unsigned blocks = (unsigned)((a.T + RT_WARPS - 1) / RT_WARPS);
  if (a.E <= 64) route_topk_kernel<LT, 2><<<blocks, RT_WARPS * 32, 0, st>>>(a);
  else if (a.E <= 128) route_topk_kernel<LT, 4><<<blocks, RT_WARPS * 32, 0, st>>>(a);
  else route_topk_kernel<LT, 8><<<blocks, RT_WARPS * 32, 0, st>>>(a);
  return cuda_ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
}

template <typename LT>
int route_bwd(const RouteBwdArgs& a, cudaStream_t st) {
  const unsigned blocks = (unsigned)((a.T + RT_WARPS - 1) / RT_WARPS);
  if (a.E <= 64) route_bwd_kernel<LT, 2><<<blocks, RT_WARPS * 32, 0, st>>>(a);
  else if (a.E <= 128) route_bwd_kernel<LT, 4><<<blocks, RT_WARPS * 32, 0, st>>>(a);
  else route_bwd_kernel<LT, 8><<<blocks, RT_WARPS * 32, 0, st>>>(a);
  return cuda_ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return type == MOE_F32 ? route_topk<float>(a, st) : route_topk<__nv_bfloat16>(a, st);
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return type == MOE_F32 ? route_bwd<float>(a, st) : route_bwd<__nv_bfloat16>(a, st);
}

}  // namespace moe
