// norm.cu -- the RMS norms before and after a block, fused with the block's gate
// and the residual's scale, and their backward (formulas in include/moe.h; the
// pages have no counterpart).
//
// HBM-bound: forward y, res -> u, n; backward dn, du, y, u -> dy, dres, every
// element once, a row in registers between its statistics and its outputs.
//
// The backward's statistics are one round of six row sums.  With a = dn w_pre,
// q = beta gate w_post y, r = 1 / rms(u) and du = d + r a - c u, c = r^3 <a, u> / d:
//   <q, du> = <q, d> + r <q, a> - c <q, u>
// so <u, u>, <a, u>, <y, y>, <q, d>, <q, a>, <q, u> give dy's mean as well.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int NB_CTAS = 148;  // backward: CTAs (row ranges), one partial row of each sum per CTA
constexpr int NV = 8;         // columns per vector

struct F8 {
  float v[NV];
};

__device__ __forceinline__ F8 ld8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ F8 ld8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const F8& r) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(r.v[2 * i], r.v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void st8(float* p, const F8& r) {
  reinterpret_cast<float4*>(p)[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
}

// Sums of N values over the CTA, the same bits in every thread.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N]) {
  __shared__ float sh[32][N];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  __syncthreads();  // the previous call's values have been read
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) sh[warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0f;
    for (int w = 0; w < nw; ++w) v[i] += sh[w][i];
  }
}

struct FwdK {
  const __nv_bfloat16* y;
  const void* res;
  const float *w_post, *gate, *w_pre;
  void* u;
  __nv_bfloat16* n;
  int64_t seq_len;  // 0: one gate row
  int d;
  float eps, alpha, beta;
};

template <typename RT, int V>
__global__ void block_norm_kernel(const FwdK a) {
  const int64_t t = blockIdx.x;
  const int nvec = a.d / NV;
  const RT* res = reinterpret_cast<const RT*>(a.res) + t * a.d;
  F8 u[V], y[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < nvec) {
      u[i] = ld8(res + c * NV);
      if (a.y) y[i] = ld8(a.y + t * a.d + c * NV);
    }
  }
  if (a.y) {
    float r1 = 1.0f;
    if (a.w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (threadIdx.x + i * blockDim.x < nvec)
#pragma unroll
          for (int j = 0; j < NV; ++j) s[0] = fmaf(y[i].v[j], y[i].v[j], s[0]);
      block_sum<1>(s);
      r1 = rsqrtf(s[0] / a.d + a.eps);
    }
    const float* gate = a.gate ? a.gate + (a.seq_len ? t / a.seq_len : 0) * a.d : nullptr;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= nvec) continue;
      F8 f;
#pragma unroll
      for (int j = 0; j < NV; ++j) f.v[j] = a.beta * r1;
      if (a.w_post) {
        const F8 w = ld8(a.w_post + c * NV);
#pragma unroll
        for (int j = 0; j < NV; ++j) f.v[j] *= w.v[j];
      }
      if (gate) {
        const F8 g = ld8(gate + c * NV);
#pragma unroll
        for (int j = 0; j < NV; ++j) f.v[j] *= g.v[j];
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) u[i].v[j] = fmaf(f.v[j], y[i].v[j], a.alpha * u[i].v[j]);
      st8(reinterpret_cast<RT*>(a.u) + t * a.d + c * NV, u[i]);
    }
  }
  if (a.n == nullptr) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (threadIdx.x + i * blockDim.x < nvec)
#pragma unroll
      for (int j = 0; j < NV; ++j) s[0] = fmaf(u[i].v[j], u[i].v[j], s[0]);
  block_sum<1>(s);
  const float r2 = rsqrtf(s[0] / a.d + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= nvec) continue;
    F8 w = ld8(a.w_pre + c * NV);
#pragma unroll
    for (int j = 0; j < NV; ++j) w.v[j] *= u[i].v[j] * r2;
    st8(a.n + t * a.d + c * NV, w);
  }
}

// Backward workspace: per CTA one row of each of the sums over its tokens --
//   post [NB_CTAS][d]  sum_t gate du y / rms(y)          -> dw_post
//   pre  [NB_CTAS][d]  sum_t dn u / rms(u)               -> dw_pre
//   seq  [NB_CTAS + sequences][d]  sum_t du y / rms(y) over the CTA's tokens of one
//        gate row, at row CTA + gate row (both grow along the tokens, so no two
//        pieces share a row)                             -> dgate
struct BwdK {
  const __nv_bfloat16 *dn, *y;
  const void *du, *u;
  const float *w_post, *gate, *w_pre;
  __nv_bfloat16* dy;
  void* dres;
  float *post, *pre, *seq;
  int64_t T, rows, seq_len;  // rows: tokens per CTA; seq_len >= 1
  int d;
  float eps, alpha, beta;
};

template <typename RT, int V>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(const BwdK a) {
  const int nvec = a.d / NV;
  const int64_t t0 = blockIdx.x * a.rows, t1 = min(t0 + a.rows, a.T);
  F8 sa[V], sp[V], sb[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < NV; ++j) sa[i].v[j] = sp[i].v[j] = sb[i].v[j] = 0.0f;
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t s = t / a.seq_len;
    const float* gate = a.gate ? a.gate + s * a.d : nullptr;
    F8 du[V], u[V], an[V], y[V], q[V], dn[V];
    float sum[6] = {0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        du[i].v[j] = u[i].v[j] = an[i].v[j] = y[i].v[j] = q[i].v[j] = dn[i].v[j] = 0.0f;
      if (c >= nvec) continue;
      const int64_t at = t * a.d + c * NV;
      if (a.du) du[i] = ld8(reinterpret_cast<const RT*>(a.du) + at);
      if (a.dn) {
        u[i] = ld8(reinterpret_cast<const RT*>(a.u) + at);
        dn[i] = ld8(a.dn + at);
        const F8 w = ld8(a.w_pre + c * NV);
#pragma unroll
        for (int j = 0; j < NV; ++j) an[i].v[j] = dn[i].v[j] * w.v[j];
      }
      if (a.y) {
        y[i] = ld8(a.y + at);
        F8 f;
#pragma unroll
        for (int j = 0; j < NV; ++j) f.v[j] = a.beta;
        if (a.w_post) {
          const F8 w = ld8(a.w_post + c * NV);
#pragma unroll
          for (int j = 0; j < NV; ++j) f.v[j] *= w.v[j];
        }
        if (gate) {
          const F8 g = ld8(gate + c * NV);
#pragma unroll
          for (int j = 0; j < NV; ++j) f.v[j] *= g.v[j];
        }
        q[i] = f;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float qy = q[i].v[j] * y[i].v[j];
        sum[0] = fmaf(u[i].v[j], u[i].v[j], sum[0]);
        sum[1] = fmaf(an[i].v[j], u[i].v[j], sum[1]);
        sum[2] = fmaf(y[i].v[j], y[i].v[j], sum[2]);
        sum[3] = fmaf(qy, du[i].v[j], sum[3]);
        sum[4] = fmaf(qy, an[i].v[j], sum[4]);
        sum[5] = fmaf(qy, u[i].v[j], sum[5]);
      }
    }
    block_sum<6>(sum);
    const float inv_d = 1.0f / a.d;
    const float r2 = rsqrtf(fmaf(sum[0], inv_d, a.eps));
    const float c2 = r2 * r2 * r2 * sum[1] * inv_d;
    const float r1 = a.w_post ? rsqrtf(fmaf(sum[2], inv_d, a.eps)) : 1.0f;
    const float c1 =
        a.w_post ? r1 * r1 * r1 * inv_d * (sum[3] + r2 * sum[4] - c2 * sum[5]) : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c >= nvec) continue;
      const int64_t at = t * a.d + c * NV;
      F8 g;
      if (gate) g = ld8(gate + c * NV);
      F8 dres, dy;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float du_j = du[i].v[j] + (a.dn ? r2 * an[i].v[j] - c2 * u[i].v[j] : 0.0f);
        dres.v[j] = a.y ? a.alpha * du_j : du_j;
        dy.v[j] = r1 * q[i].v[j] * du_j - c1 * y[i].v[j];
        const float x = du_j * (r1 * y[i].v[j]);
        sa[i].v[j] += x;
        sp[i].v[j] += gate ? g.v[j] * x : x;
        sb[i].v[j] += dn[i].v[j] * (r2 * u[i].v[j]);
      }
      st8(reinterpret_cast<RT*>(a.dres) + at, dres);
      if (a.y) st8(a.dy + at, dy);
    }
    if (a.seq && (t + 1 == t1 || (t + 1) / a.seq_len != s)) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nvec) st8(a.seq + ((int64_t)blockIdx.x + s) * a.d + c * NV, sa[i]);
#pragma unroll
        for (int j = 0; j < NV; ++j) sa[i].v[j] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c >= nvec) continue;
    if (a.post) st8(a.post + (int64_t)blockIdx.x * a.d + c * NV, sp[i]);
    if (a.pre) st8(a.pre + (int64_t)blockIdx.x * a.d + c * NV, sb[i]);
  }
}

struct FinK {
  const float *post, *pre, *seq, *w_post;
  float *dw_post, *dw_pre, *dgate;
  int64_t T, rows, seq_len;
  int ctas, d, accumulate;
  float beta;
};

// Column sums of the CTAs' rows: job 0 dw_post, 1 dw_pre, 2 + s dgate row s.
// 32 columns x 8 strands of rows, the strands added in order.
__global__ void __launch_bounds__(256) block_norm_bwd_finish(const FinK a) {
  __shared__ float sh[8][32];
  const int x = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int cols = (a.d + 31) / 32;
  const int64_t job = blockIdx.x / cols;
  const int c = (int)(blockIdx.x - job * cols) * 32 + x;
  const float* src;
  float* dst;
  int64_t r0 = 0, r1 = a.ctas;
  float f = 1.0f;
  if (job == 0) {
    src = a.post;
    dst = a.dw_post;
    f = a.beta;
  } else if (job == 1) {
    src = a.pre;
    dst = a.dw_pre;
  } else {
    const int64_t s = job - 2;
    const int64_t last = min((s + 1) * a.seq_len, a.T) - 1;
    r0 = s * a.seq_len / a.rows + s;
    r1 = last / a.rows + s + 1;
    src = a.seq;
    dst = a.dgate ? a.dgate + s * a.d : nullptr;
    f = a.beta * (a.w_post && c < a.d ? a.w_post[c] : 1.0f);
  }
  if (dst == nullptr) return;
  float v = 0.0f;
  if (c < a.d)
    for (int64_t r = r0 + strand; r < r1; r += 8) v += src[r * a.d + c];
  sh[strand][x] = v;
  __syncthreads();
  if (strand == 0 && c < a.d) {
    for (int i = 1; i < 8; ++i) v += sh[i][x];
    dst[c] = a.accumulate ? dst[c] + f * v : f * v;
  }
}

int64_t gate_rows(const moe_dims& dm, const moe_norm_cfg& c) {
  return c.seq_len && dm.T ? (dm.T + c.seq_len - 1) / c.seq_len : 1;
}

template <typename RT, int V>
void fwd(const FwdK& k, int64_t T, int threads, cudaStream_t st) {
  block_norm_kernel<RT, V><<<(unsigned)T, threads, 0, st>>>(k);
}

template <typename RT>
void fwd_any(const FwdK& k, int64_t T, cudaStream_t st) {
  const int nvec = k.d / NV;
  auto threads = [&](int v) { return ((nvec + v - 1) / v + 31) / 32 * 32; };
  if (nvec <= 512) fwd<RT, 1>(k, T, threads(1), st);
  else if (nvec <= 1024) fwd<RT, 2>(k, T, threads(2), st);
  else fwd<RT, 4>(k, T, threads(4), st);
}

template <typename RT>
void bwd_any(const BwdK& k, unsigned ctas, cudaStream_t st) {
  const int nvec = k.d / NV;
  auto threads = [&](int v) { return ((nvec + v - 1) / v + 31) / 32 * 32; };
  if (nvec <= 512) block_norm_bwd_kernel<RT, 1><<<ctas, threads(1), 0, st>>>(k);
  else if (nvec <= 1024) block_norm_bwd_kernel<RT, 2><<<ctas, threads(2), 0, st>>>(k);
  else block_norm_bwd_kernel<RT, 4><<<ctas, threads(4), 0, st>>>(k);
}

}  // namespace

size_t norm_ws_bytes(const moe_dims& dm, const moe_norm_cfg& c) {
  return align_up((size_t)(3 * NB_CTAS + gate_rows(dm, c)) * dm.d * sizeof(float), 256);
}

int launch_block_norm(const moe_dims& dm, const moe_norm_cfg& c, int res_type, const NormArgs& a,
                      void* stream) {
  if (dm.T == 0) return MOE_OK;
  FwdK k{};
  k.y = reinterpret_cast<const __nv_bfloat16*>(a.y);
  k.res = a.res;
  k.w_post = a.w_post;
  k.gate = a.gate;
  k.w_pre = a.w_pre;
  k.u = a.u;
  k.n = reinterpret_cast<__nv_bfloat16*>(a.n);
  k.seq_len = c.seq_len;
  k.d = dm.d;
  k.eps = c.eps;
  k.alpha = c.res_scale;
  k.beta = c.block_scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (res_type == MOE_F32) fwd_any<float>(k, dm.T, st);
  else fwd_any<__nv_bfloat16>(k, dm.T, st);
  return cuda_ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
}

int launch_block_norm_bwd(const moe_dims& dm, const moe_norm_cfg& c, int res_type,
                          const NormArgs& a, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t seqs = gate_rows(dm, c);
  if ((2 + seqs) * ((dm.d + 31) / 32) >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
  BwdK k{};
  k.dn = reinterpret_cast<const __nv_bfloat16*>(a.dn);
  k.y = reinterpret_cast<const __nv_bfloat16*>(a.y);
  k.du = a.du;
  k.u = a.res;
  k.w_post = a.w_post;
  k.gate = a.gate;
  k.w_pre = a.w_pre;
  k.dy = reinterpret_cast<__nv_bfloat16*>(a.dy);
  k.dres = a.dres;
  float* ws = reinterpret_cast<float*>(a.ws);
  k.post = a.dw_post ? ws : nullptr;
  k.pre = a.dw_pre ? ws + (size_t)NB_CTAS * dm.d : nullptr;
  k.seq = a.dgate ? ws + (size_t)2 * NB_CTAS * dm.d : nullptr;
  k.T = dm.T;
  k.rows = (dm.T + NB_CTAS - 1) / NB_CTAS;
  k.seq_len = c.seq_len ? c.seq_len : (dm.T ? dm.T : 1);
  k.d = dm.d;
  k.eps = c.eps;
  k.alpha = c.res_scale;
  k.beta = c.block_scale;
  const unsigned ctas = dm.T ? (unsigned)((dm.T + k.rows - 1) / k.rows) : 0;
  if (ctas) {
    if (res_type == MOE_F32) bwd_any<float>(k, ctas, st);
    else bwd_any<__nv_bfloat16>(k, ctas, st);
    if (!cuda_ok(cudaGetLastError())) return MOE_ERR_CUDA;
  }
  if (!a.dw_post && !a.dw_pre && !a.dgate) return MOE_OK;
  FinK f{};
  f.post = k.post;
  f.pre = k.pre;
  f.seq = k.seq;
  f.w_post = a.w_post;
  f.dw_post = a.dw_post;
  f.dw_pre = a.dw_pre;
  f.dgate = a.dgate;
  f.T = dm.T;
  f.rows = k.rows ? k.rows : 1;
  f.seq_len = k.seq_len;
  f.ctas = (int)ctas;
  f.d = dm.d;
  f.accumulate = a.accumulate;
  f.beta = a.y ? c.block_scale : 1.0f;
  block_norm_bwd_finish<<<(unsigned)((2 + seqs) * ((dm.d + 31) / 32)), 256, 0, st>>>(f);
  return cuda_ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
