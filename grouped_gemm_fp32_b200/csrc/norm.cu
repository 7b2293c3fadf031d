// norm.cu -- the RMS norms before and after a block, fused with the block's gate
// and the residual's scale, and their backward (formulas in include/moe.h; the
// pages have no counterpart).
//
// HBM-bound: forward y, res -> u, n; backward dn, du, y, u -> dy, dres, every
// element once.  Persistent CTAs walk a contiguous range of rows each, a row spread
// over the CTA's threads, eight columns a vector.  Rows come in by cp.async into a ring
// in shared memory, several rows ahead; a thread copies and reads its own columns only,
// so a row costs one barrier a statistic and none for its data.  The weights stay in
// registers (rows of up to 8192 columns), and so do the backward's sums over tokens.
//
// The backward's statistics are one round of six row sums.  With a = dn w_pre,
// q = beta gate w_post y, r = 1 / rms(u) and du = d + r a - c u, c = r^3 <a, u> / d:
//   <q, du> = <q, d> + r <q, a> - c <q, u>
// so <u, u>, <a, u>, <y, y>, <q, d>, <q, a>, <q, u> give dy's mean as well.
#include <atomic>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "moe_internal.cuh"
#include "sm100.cuh"

namespace moe {
namespace {

constexpr int NB_SMS = 148;       // SMs of a B200; CTAs are a multiple of it
constexpr int NB_STAGES = 8;      // most rows in a ring
constexpr int NB_SMEM = 226 * 1024;  // an SM's shared memory for its CTAs' rings
constexpr int NV = 8;             // columns per vector

// How rows of d columns are spread over a CTA: V vectors a thread, and how many CTAs
// share an SM (512 threads an SM; fewer threads than that leave the copies in flight, not
// the arithmetic, to fill it).
struct Shape {
  int v, threads, per_sm;
};
Shape shape_of(int d) {
  const int nvec = d / NV;
  Shape s;
  s.v = nvec <= 256 ? 1 : nvec <= 1024 ? 2 : 4;
  s.threads = ((nvec + s.v - 1) / s.v + 31) / 32 * 32;
  s.per_sm = 512 / s.threads;
  if (s.per_sm > 16) s.per_sm = 16;
  return s;
}

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

// Sums of N values over the CTA, the same bits in every thread.  Calls alternate between
// two halves of sh [2][16][N], so one barrier a call is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* sh, int& half) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  float* mine = sh + half * 16 * N;
  half ^= 1;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) mine[warp * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = mine[i];
  for (int w = 1; w < nw; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += mine[w * N + i];
}

__device__ __forceinline__ void cp16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most n of this thread's copy groups are still in flight.
__device__ __forceinline__ void cp_wait(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
  }
}

// One matrix's row in a ring stage: 16 bytes a vector in bf16, two pieces of 16 in FP32,
// the first pieces of all vectors before the second ones.
__device__ __forceinline__ void cp_row(uint4* st, int nvec, int c, const __nv_bfloat16* g) {
  cp16(st + c, g);
}
__device__ __forceinline__ void cp_row(uint4* st, int nvec, int c, const float* g) {
  cp16(st + c, g);
  cp16(st + nvec + c, g + 4);
}
__device__ __forceinline__ F8 rd_row(const uint4* st, int nvec, int c, const __nv_bfloat16*) {
  return ld8(reinterpret_cast<const __nv_bfloat16*>(st + c));
}
__device__ __forceinline__ F8 rd_row(const uint4* st, int nvec, int c, const float*) {
  const float4 a = *reinterpret_cast<const float4*>(st + c);
  const float4 b = *reinterpret_cast<const float4*>(st + nvec + c);
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

struct FwdK {
  const __nv_bfloat16* y;
  const void* res;
  const float *w_post, *gate, *w_pre;
  void* u;
  __nv_bfloat16* n;
  int64_t T, rows, seq_len;  // rows: tokens per CTA; seq_len >= 1
  int d, stages;
  float eps, alpha, beta;
};

// beta gate w_post of a vector (w_post and gate may be NULL).
__device__ __forceinline__ F8 post_factor(const float* w_post, const float* gate, float beta,
                                          int c) {
  F8 f;
#pragma unroll
  for (int j = 0; j < NV; ++j) f.v[j] = beta;
  if (w_post) {
    const F8 w = ld8(w_post + c * NV);
#pragma unroll
    for (int j = 0; j < NV; ++j) f.v[j] *= w.v[j];
  }
  if (gate) {
    const F8 g = ld8(gate + c * NV);
#pragma unroll
    for (int j = 0; j < NV; ++j) f.v[j] *= g.v[j];
  }
  return f;
}

template <typename RT, int V, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) block_norm_kernel(const FwdK a) {
  constexpr bool KEEP = V <= 2;  // the weights in registers; else read again every row
  constexpr int R = sizeof(RT) / 2;
  extern __shared__ uint4 ring[];
  __shared__ float sh[2 * 16];
  int half = 0;
  const int nvec = a.d / NV, tid = threadIdx.x, nt = blockDim.x;
  const int64_t t0 = blockIdx.x * a.rows, t1 = min(t0 + a.rows, a.T);
  const int S = a.stages, row_v = (1 + R) * nvec;  // a stage: y, then res
  const RT* res = reinterpret_cast<const RT*>(a.res);
  RT* u_out = reinterpret_cast<RT*>(a.u);
  int put = 0, get = 0;  // ring stages of the next row to copy and to read
  auto issue = [&](int64_t t) {
    if (t < t1) {
      uint4* st = ring + (size_t)put * row_v;
      put = put + 1 == S ? 0 : put + 1;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        if (c >= nvec) continue;
        const int64_t at = t * a.d + c * NV;
        if (a.y) cp_row(st, nvec, c, a.y + at);
        cp_row(st + nvec, nvec, c, res + at);
      }
    }
    cp_commit();
  };
  for (int s = 0; s + 1 < S; ++s) issue(t0 + s);
  F8 f[KEEP ? V : 1], wp[KEEP ? V : 1];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (a.w_pre && tid + i * nt < nvec) wp[i] = ld8(a.w_pre + (tid + i * nt) * NV);
  }
  int64_t seq_end = t0;  // first token past the gate row that f holds
  const float* gate = nullptr;
  for (int64_t t = t0; t < t1; ++t) {
    if (t >= seq_end) {
      const int64_t s = t / a.seq_len;
      seq_end = (s + 1) * a.seq_len;
      if (a.gate) gate = a.gate + s * a.d;
      if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (a.y && tid + i * nt < nvec)
            f[i] = post_factor(a.w_post, gate, a.beta, tid + i * nt);
      }
    }
    if (S == 1) {
      __syncthreads();
      issue(t);
    }
    cp_wait(S > 1 ? S - 2 : 0);
    const uint4* st = ring + (size_t)get * row_v;
    get = get + 1 == S ? 0 : get + 1;
    F8 u[V];
    float s[1] = {0.0f};
    if (a.y) {
      F8 y[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (tid + i * nt < nvec) {
          y[i] = rd_row(st, nvec, tid + i * nt, a.y);
#pragma unroll
          for (int j = 0; j < NV; ++j) s[0] = fmaf(y[i].v[j], y[i].v[j], s[0]);
        }
      float r1 = 1.0f;
      if (a.w_post) {
        block_sum<1>(s, sh, half);
        r1 = rsqrtf(s[0] / a.d + a.eps);
      }
      s[0] = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        if (c >= nvec) continue;
        u[i] = rd_row(st + nvec, nvec, c, res);
        const F8 g = KEEP ? f[KEEP ? i : 0] : post_factor(a.w_post, gate, a.beta, c);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          u[i].v[j] = fmaf(g.v[j] * r1, y[i].v[j], a.alpha * u[i].v[j]);
          s[0] = fmaf(u[i].v[j], u[i].v[j], s[0]);
        }
        st8(u_out + t * a.d + c * NV, u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (tid + i * nt < nvec) {
          u[i] = rd_row(st + nvec, nvec, tid + i * nt, res);
#pragma unroll
          for (int j = 0; j < NV; ++j) s[0] = fmaf(u[i].v[j], u[i].v[j], s[0]);
        }
    }
    // a copy refills the stage of the row before this one: every thread has passed a
    // barrier since it read that
    if (a.n) {
      block_sum<1>(s, sh, half);
      if (S > 1) issue(t + S - 1);
      const float r2 = rsqrtf(s[0] / a.d + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        if (c >= nvec) continue;
        F8 w = KEEP ? wp[KEEP ? i : 0] : ld8(a.w_pre + c * NV);
#pragma unroll
        for (int j = 0; j < NV; ++j) w.v[j] *= u[i].v[j] * r2;
        st8(a.n + t * a.d + c * NV, w);
      }
    } else {
      if (!a.w_post) __syncthreads();  // as a statistic's barrier
      if (S > 1) issue(t + S - 1);
    }
  }
}

// Backward workspace, with C the CTAs: per CTA one row of each of the sums over its
// tokens --
//   post [C][d]  sum_t gate du y / rms(y)          -> dw_post
//   pre  [C][d]  sum_t dn u / rms(u)               -> dw_pre
//   seq  [C + sequences][d]  sum_t du y / rms(y) over the CTA's tokens of one gate row,
//        at row CTA + gate row (both grow along the tokens, so no two pieces share a
//        row)                                      -> dgate
struct BwdK {
  const __nv_bfloat16 *dn, *y;
  const void *du, *u;
  const float *w_post, *gate, *w_pre;
  __nv_bfloat16* dy;
  void* dres;
  float *post, *pre, *seq;
  int64_t T, rows, seq_len;  // rows: tokens per CTA; seq_len >= 1
  int d, stages;
  float eps, alpha, beta;
};

template <typename RT, int V, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) block_norm_bwd_kernel(const BwdK a) {
  constexpr bool KEEP = V <= 2;
  constexpr int R = sizeof(RT) / 2;
  extern __shared__ uint4 ring[];
  __shared__ float sh[2 * 16 * 6];
  int half = 0;
  const int nvec = a.d / NV, tid = threadIdx.x, nt = blockDim.x;
  const int64_t t0 = blockIdx.x * a.rows, t1 = min(t0 + a.rows, a.T);
  const int S = a.stages, row_v = (2 + 2 * R) * nvec;  // a stage: dn, y, dres_out, u
  const RT* du_in = reinterpret_cast<const RT*>(a.du);
  const RT* u_in = reinterpret_cast<const RT*>(a.u);
  RT* dres_out = reinterpret_cast<RT*>(a.dres);
  int put = 0, get = 0;  // ring stages of the next row to copy and to read
  auto issue = [&](int64_t t) {
    if (t < t1) {
      uint4* st = ring + (size_t)put * row_v;
      put = put + 1 == S ? 0 : put + 1;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        if (c >= nvec) continue;
        const int64_t at = t * a.d + c * NV;
        if (a.dn) {
          cp_row(st, nvec, c, a.dn + at);
          cp_row(st + (2 + R) * nvec, nvec, c, u_in + at);
        }
        if (a.y) cp_row(st + nvec, nvec, c, a.y + at);
        if (a.du) cp_row(st + 2 * nvec, nvec, c, du_in + at);
      }
    }
    cp_commit();
  };
  // matrices that are not there read as zeros: no copy ever writes their part of the ring
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * nt;
      if (c >= nvec) continue;
      uint4* st = ring + (size_t)s * row_v;
      const uint4 z = make_uint4(0, 0, 0, 0);
      if (!a.dn) {
        st[c] = z;
#pragma unroll
        for (int r = 0; r < R; ++r) st[(2 + R + r) * nvec + c] = z;
      }
      if (!a.y) st[nvec + c] = z;
      if (!a.du) {
#pragma unroll
        for (int r = 0; r < R; ++r) st[(2 + r) * nvec + c] = z;
      }
    }
  for (int s = 0; s + 1 < S; ++s) issue(t0 + s);
  F8 sa[V], sb[V], f[KEEP ? V : 1], wp[KEEP ? V : 1];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < NV; ++j) sa[i].v[j] = sb[i].v[j] = 0.0f;
  const F8 zero = sa[0];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      wp[i] = a.dn && tid + i * nt < nvec ? ld8(a.w_pre + (tid + i * nt) * NV) : zero;
  }
  const float inv_d = 1.0f / a.d, alpha = a.y ? a.alpha : 1.0f;
  int64_t seq_end = t0, seq = 0;  // the gate row that f holds, and the first token past it
  const float* gate = nullptr;
  bool flushed = false;  // post holds the sums of earlier gate rows
  for (int64_t t = t0; t < t1; ++t) {
    if (t >= seq_end) {
      seq = t / a.seq_len;
      seq_end = (seq + 1) * a.seq_len;
      if (a.gate) gate = a.gate + seq * a.d;
      if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          f[i] = a.y && tid + i * nt < nvec ? post_factor(a.w_post, gate, a.beta, tid + i * nt)
                                            : zero;
      }
    }
    if (S == 1) {
      __syncthreads();
      issue(t);
    }
    cp_wait(S > 1 ? S - 2 : 0);
    const uint4* st = ring + (size_t)get * row_v;
    get = get + 1 == S ? 0 : get + 1;
    float sum[6] = {0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * nt;
      if (c >= nvec) continue;
      const F8 dn = rd_row(st, nvec, c, a.dn), y = rd_row(st + nvec, nvec, c, a.y);
      const F8 du = rd_row(st + 2 * nvec, nvec, c, du_in);
      const F8 u = rd_row(st + (2 + R) * nvec, nvec, c, u_in);
      F8 g, w;
      if constexpr (KEEP) {
        g = f[i];
        w = wp[i];
      } else {
        g = a.y ? post_factor(a.w_post, gate, a.beta, c) : zero;
        w = a.dn ? ld8(a.w_pre + c * NV) : zero;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float an = dn.v[j] * w.v[j], qy = g.v[j] * y.v[j];
        sum[0] = fmaf(u.v[j], u.v[j], sum[0]);
        sum[1] = fmaf(an, u.v[j], sum[1]);
        sum[2] = fmaf(y.v[j], y.v[j], sum[2]);
        sum[3] = fmaf(qy, du.v[j], sum[3]);
        sum[4] = fmaf(qy, an, sum[4]);
        sum[5] = fmaf(qy, u.v[j], sum[5]);
      }
    }
    block_sum<6>(sum, sh, half);
    // the stage of the row before this one: every thread has passed a barrier since it read it
    if (S > 1) issue(t + S - 1);
    const float r2 = a.dn ? rsqrtf(fmaf(sum[0], inv_d, a.eps)) : 0.0f;
    const float c2 = r2 * r2 * r2 * sum[1] * inv_d;
    const float r1 = a.w_post ? rsqrtf(fmaf(sum[2], inv_d, a.eps)) : 1.0f;
    const float c1 =
        a.w_post ? r1 * r1 * r1 * inv_d * (sum[3] + r2 * sum[4] - c2 * sum[5]) : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * nt;
      if (c >= nvec) continue;
      const F8 dn = rd_row(st, nvec, c, a.dn), y = rd_row(st + nvec, nvec, c, a.y);
      const F8 du = rd_row(st + 2 * nvec, nvec, c, du_in);
      const F8 u = rd_row(st + (2 + R) * nvec, nvec, c, u_in);
      F8 g, w, dres, dy;
      if constexpr (KEEP) {
        g = f[i];
        w = wp[i];
      } else {
        g = a.y ? post_factor(a.w_post, gate, a.beta, c) : zero;
        w = a.dn ? ld8(a.w_pre + c * NV) : zero;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float v = du.v[j] + (r2 * (dn.v[j] * w.v[j]) - c2 * u.v[j]);
        dres.v[j] = alpha * v;
        const float x = r1 * v;
        dy.v[j] = g.v[j] * x - c1 * y.v[j];
        sa[i].v[j] = fmaf(x, y.v[j], sa[i].v[j]);
        sb[i].v[j] = fmaf(dn.v[j], r2 * u.v[j], sb[i].v[j]);
      }
      const int64_t at = t * a.d + c * NV;
      st8(dres_out + at, dres);
      if (a.y) st8(a.dy + at, dy);
    }
    if (t + 1 == t1 || t + 1 == seq_end) {  // the gate row's sums are complete here
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = tid + i * nt;
        if (c >= nvec) continue;
        if (a.seq) st8(a.seq + ((int64_t)blockIdx.x + seq) * a.d + c * NV, sa[i]);
        if (a.post) {
          float* p = a.post + (int64_t)blockIdx.x * a.d + c * NV;
          F8 v = flushed ? ld8(p) : zero;
          const F8 g = gate ? ld8(gate + c * NV) : zero;
#pragma unroll
          for (int j = 0; j < NV; ++j) v.v[j] += gate ? g.v[j] * sa[i].v[j] : sa[i].v[j];
          st8(p, v);
        }
        sa[i] = zero;
      }
      flushed = true;
    }
  }
  if (a.pre)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (tid + i * nt < nvec) st8(a.pre + (int64_t)blockIdx.x * a.d + (tid + i * nt) * NV, sb[i]);
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

// CTAs of a launch over T rows and the rows each takes.
int64_t split_rows(int64_t T, int d, int64_t* rows) {
  const int64_t most = (int64_t)NB_SMS * shape_of(d).per_sm;
  *rows = T ? (T + most - 1) / most : 1;
  return (T + *rows - 1) / *rows;
}

// Raises a kernel's shared-memory limit, once per device (a bit of `ready` each).
template <typename K>
bool opt_in(void (*kernel)(const K), std::atomic<uint64_t>& ready) {
  int dev = 0;
  if (!cuda_ok(cudaGetDevice(&dev))) return false;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (ready.load(std::memory_order_relaxed) & bit) return true;
  if (!cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    NB_SMEM - 1536)))
    return false;
  ready.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// Launch on rows of `pieces` 16-byte pieces a vector: the ring takes what its CTA's share
// of the SM's shared memory holds, the CTA's rows at most.
template <typename K>
int launch_rows(void (*kernel)(const K), std::atomic<uint64_t>& ready, K k, int pieces,
                int64_t ctas, cudaStream_t st) {
  const Shape s = shape_of(k.d);
  const int64_t stage = (int64_t)pieces * (k.d / NV) * 16;
  int64_t n = (NB_SMEM / s.per_sm - 1536) / stage;  // 1 KB a CTA and the static part beside it
  if (n > NB_STAGES) n = NB_STAGES;
  if (n > k.rows + 1) n = k.rows + 1;
  if (n < 1) n = 1;
  k.stages = (int)n;
  const int bytes = (int)(n * stage);
  if (!opt_in(kernel, ready)) return MOE_ERR_CUDA;
  kernel<<<(unsigned)ctas, s.threads, bytes, st>>>(k);
  return cuda_ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
}

template <typename RT>
int fwd(const FwdK& k, int64_t ctas, cudaStream_t st) {
  const Shape s = shape_of(k.d);
  const int pieces = 1 + sizeof(RT) / 2;
  static std::atomic<uint64_t> ready[4];
  if (s.v == 1) return launch_rows(block_norm_kernel<RT, 1, 256>, ready[0], k, pieces, ctas, st);
  if (s.v == 2 && s.threads <= 256)
    return launch_rows(block_norm_kernel<RT, 2, 256>, ready[1], k, pieces, ctas, st);
  if (s.v == 2) return launch_rows(block_norm_kernel<RT, 2, 512>, ready[2], k, pieces, ctas, st);
  return launch_rows(block_norm_kernel<RT, 4, 512>, ready[3], k, pieces, ctas, st);
}

template <typename RT>
int bwd(const BwdK& k, int64_t ctas, cudaStream_t st) {
  const Shape s = shape_of(k.d);
  const int pieces = 2 + 2 * (sizeof(RT) / 2);
  static std::atomic<uint64_t> ready[4];
  if (s.v == 1) return launch_rows(block_norm_bwd_kernel<RT, 1, 256>, ready[0], k, pieces, ctas, st);
  if (s.v == 2 && s.threads <= 256)
    return launch_rows(block_norm_bwd_kernel<RT, 2, 256>, ready[1], k, pieces, ctas, st);
  if (s.v == 2) return launch_rows(block_norm_bwd_kernel<RT, 2, 512>, ready[2], k, pieces, ctas, st);
  return launch_rows(block_norm_bwd_kernel<RT, 4, 512>, ready[3], k, pieces, ctas, st);
}

}  // namespace

size_t norm_ws_bytes(const moe_dims& dm, const moe_norm_cfg& c) {
  int64_t rows;
  const int64_t ctas = split_rows(dm.T, dm.d, &rows);
  return align_up((size_t)(3 * ctas + gate_rows(dm, c)) * dm.d * sizeof(float), 256);
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
  k.T = dm.T;
  const int64_t ctas = split_rows(dm.T, dm.d, &k.rows);
  k.seq_len = c.seq_len ? c.seq_len : dm.T;
  k.d = dm.d;
  k.eps = c.eps;
  k.alpha = c.res_scale;
  k.beta = c.block_scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return res_type == MOE_F32 ? fwd<float>(k, ctas, st) : fwd<__nv_bfloat16>(k, ctas, st);
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
  const int64_t ctas = split_rows(dm.T, dm.d, &k.rows);
  k.post = a.dw_post ? ws : nullptr;
  k.pre = a.dw_pre ? ws + (size_t)ctas * dm.d : nullptr;
  k.seq = a.dgate ? ws + (size_t)2 * ctas * dm.d : nullptr;
  k.T = dm.T;
  k.seq_len = c.seq_len ? c.seq_len : (dm.T ? dm.T : 1);
  k.d = dm.d;
  k.eps = c.eps;
  k.alpha = c.res_scale;
  k.beta = c.block_scale;
  if (ctas) {
    const int rc =
        res_type == MOE_F32 ? bwd<float>(k, ctas, st) : bwd<__nv_bfloat16>(k, ctas, st);
    if (rc != MOE_OK) return rc;
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
  f.rows = k.rows;
  f.seq_len = k.seq_len;
  f.ctas = (int)ctas;
  f.d = dm.d;
  f.accumulate = a.accumulate;
  f.beta = a.y ? c.block_scale : 1.0f;
  block_norm_bwd_finish<<<(unsigned)((2 + seqs) * ((dm.d + 31) / 32)), 256, 0, st>>>(f);
  return cuda_ok(cudaGetLastError()) ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
