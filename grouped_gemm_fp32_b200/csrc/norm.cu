// norm.cu -- the RMS norms before and after a block, fused with the block's gate
// and the residual's scale, and their backward (formulas in include/moe.h; the
// pages have no counterpart).
//
// HBM-bound: forward y, res -> u, n; backward dn, du, y, u -> dy, dres, every
// element once.  Persistent CTAs walk a contiguous range of rows each, a row spread
// over the CTA's threads, eight columns a vector.  Rows come in by cp.async into a ring
// in shared memory, several rows ahead; a thread reads what it copied itself (bf16 rows
// beside an FP32 residual: what its warp copied), so a row costs one barrier a statistic and
// none for its data.  The weights stay in registers (rows of up to 8192 columns), and so do
// the backward's sums over tokens.
//
// Measured, of the 6458 GB/s of a copy: 8192 x 4096 forward, bf16 residual, 51 us (0.81);
// 16384 x 4096 backward with gates 146 us (0.86); with an FP32 residual 142 us (0.88) and
// 202 us (0.93).
//
// A row's sums are means: 1 / d is taken of sums of at most 256 products (a thread's, or eight
// lanes') before they are added up, so that rows of values up to 1e18 stay in FP32's range at
// any width.
//
// The backward's statistics are one round of six row sums.  With a = dn w_pre, r2 = 1 / rms(u),
// uh = r2 u, m2 = mean(a uh), v = dres_out + r2 (a - m2 uh) the gradient of u, and with
// g = beta gate w_post, q = g y, r1 = 1 / rms(y), yh = r1 y, m1 = mean(g v yh):
//   dy = r1 (g v - m1 yh),   m1 = r1 (mean(q dres_out) + r2 (mean(q a) - m2 r2 mean(q u)))
// so u u, a u, y y, q dres_out, q a and q u are all that is summed.  Factors r1^3 and r2^3 in
// place of uh and yh would save two products, and leave FP32's range for rows from 1e13 on and
// below 1e-12.
#include <algorithm>
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
// the arithmetic, to fill it).  Two vectors a thread halve what a row costs beside its
// arithmetic and double the rows in work on an SM.  Forward that pays from two vectors a
// lane on: 16384 rows of 512 columns 10.4 instead of 15.4 us, 1024 22 instead of 30, 1536 39
// instead of 56.  The backward has more arithmetic and registers, and more CTAs, of which few
// rows, and rows of many gates, feel the column sums: up to 1024 columns one vector is faster
// at any number of rows (16384 of 768 42 instead of 45 us, 2000 of 1024 13 instead of 16).  To
// 2048 columns the wider the rows the fewer of them it takes; one vector against two, a gate
// row for all: 1088 columns 11.7 / 13.2 us for 1000 rows, 13.9 / 14.9 for 2000, 60 / 59 for
// 16384; 1536 columns 13.5 / 14.0, 18.7 / 16.0, 71 / 58; 2048 columns 15.8 / 14.3, 19.2 / 16.7,
// 82 / 76 (11.3 / 13.6 for 500).  With a gate row for 130 tokens one vector stays ahead: 2048
// columns 13.8 / 17.2, 19.6 / 25.3, 95 / 145.  1024 rows stand between the two.
struct Shape {
  int v, threads, per_sm;
};
Shape shape_of(int64_t T, int d, bool bwd) {
  const int nvec = d / NV;
  Shape s;
  s.v = nvec <= (!bwd ? 32 : T < 1024 ? 256 : 128) ? 1 : nvec <= 1024 ? 2 : 4;
  s.threads = ((nvec + s.v - 1) / s.v + 31) / 32 * 32;
  s.per_sm = 512 / s.threads;
  if (s.per_sm > 16) s.per_sm = 16;
  return s;
}

// Two FP32 values in a register pair, for the paired FP32 instructions (each half rounds
// like the single instruction).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
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
__device__ __forceinline__ float sum2(f32x2 v) {
  const float2 f = halves(v);
  return f.x + f.y;
}

// Eight columns.
struct F8 {
  f32x2 v[NV / 2];
};

__device__ __forceinline__ F8 splat(float f) {
  F8 r;
#pragma unroll
  for (int i = 0; i < NV / 2; ++i) r.v[i] = both(f);
  return r;
}
__device__ __forceinline__ F8 from_bf16(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  return r;
}
// Which eight columns of a row a thread has as vector c: [a, a + 4) and [b, b + 4).  With a
// bf16 residual they are the 16 bytes of vector c.  With an FP32 one they lie in the two
// halves of the columns of the warp's vectors, so that a warp's 16-byte accesses to FP32
// rows and its 8-byte accesses to bf16 ones are each contiguous (side by side, the eight
// would be half sectors of the L2 apart: 16384 x 7168 took 303 us forward).
struct Cols {
  int a, b;
};
template <bool SPLIT>
__device__ __forceinline__ Cols cols_of(int c, int nvec) {
  if constexpr (!SPLIT) return {c * NV, c * NV + 4};
  const int l = c & 31, base = c - l;
  const int a = base * NV + 4 * l;
  return {a, a + 4 * min(32, nvec - base)};
}

__device__ __forceinline__ F8 ld8(const float* p, Cols o) {
  const float4 a = *reinterpret_cast<const float4*>(p + o.a);
  const float4 b = *reinterpret_cast<const float4*>(p + o.b);
  return F8{{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
}
template <bool SPLIT>
__device__ __forceinline__ F8 ld8(const __nv_bfloat16* p, Cols o) {
  if constexpr (!SPLIT) return from_bf16(*reinterpret_cast<const uint4*>(p + o.a));
  const uint2 a = *reinterpret_cast<const uint2*>(p + o.a);
  const uint2 b = *reinterpret_cast<const uint2*>(p + o.b);
  return from_bf16(make_uint4(a.x, a.y, b.x, b.y));
}
template <bool SPLIT>
__device__ __forceinline__ F8 ld8(const float* p, Cols o) {
  return ld8(p, o);
}
__device__ __forceinline__ void st8(float* p, Cols o, const F8& r) {
  const float2 a = halves(r.v[0]), b = halves(r.v[1]), c = halves(r.v[2]), d = halves(r.v[3]);
  *reinterpret_cast<float4*>(p + o.a) = make_float4(a.x, a.y, b.x, b.y);
  *reinterpret_cast<float4*>(p + o.b) = make_float4(c.x, c.y, d.x, d.y);
}
template <bool SPLIT>
__device__ __forceinline__ void st8(__nv_bfloat16* p, Cols o, const F8& r) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __float22bfloat162_rn(halves(r.v[i]));
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if constexpr (!SPLIT) {
    *reinterpret_cast<uint4*>(p + o.a) = u;
  } else {
    *reinterpret_cast<uint2*>(p + o.a) = make_uint2(u.x, u.y);
    *reinterpret_cast<uint2*>(p + o.b) = make_uint2(u.z, u.w);
  }
}
template <bool SPLIT>
__device__ __forceinline__ void st8(float* p, Cols o, const F8& r) {
  st8(p, o, r);
}

constexpr int MAX_WARPS = 16;  // of a CTA

// Sum over the CTA, the same bits in every thread.  Calls alternate between two halves of
// sh [2][MAX_WARPS] (zero beyond the CTA's warps), so one barrier a call is enough.
__device__ __forceinline__ float block_sum1(float v, float* sh, int& half) {
  float* mine = sh + half * MAX_WARPS;
  half ^= 1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  const int quads = (int)(blockDim.x + 127) >> 7;
  for (int i = 0; i < quads; ++i) {
    const float4 f = reinterpret_cast<const float4*>(mine)[i];
    s += (f.x + f.y) + (f.z + f.w);
  }
  return s;
}

// Six sums over the CTA, by inv_d.  In a warp the lanes halve the values they carry at every step
// (3 + 2 + 1 + 1 + 1 shuffles where six sums take 30): lanes 4 i .. 4 i + 3 end with value
// i (values 3 and 7 are not used).  sh [2][MAX_WARPS][8] as above; every warp then adds the
// warps' rows and hands all six to every lane.
__device__ __forceinline__ void block_mean6(float (&v)[6], float inv_d, float* sh, int& half) {
  constexpr unsigned ALL = 0xffffffffu;
  float* mine = sh + half * MAX_WARPS * 8;
  half ^= 1;
  const int lane = threadIdx.x & 31;
  const bool up16 = lane & 16, up8 = lane & 8, up4 = lane & 4;
  float w[4];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float keep = up16 ? v[3 + i] : v[i], give = up16 ? v[i] : v[3 + i];
    w[i] = keep + __shfl_xor_sync(ALL, give, 16);
  }
  w[3] = 0.0f;
  float x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = up8 ? w[2 + i] : w[i], give = up8 ? w[i] : w[2 + i];
    x[i] = keep + __shfl_xor_sync(ALL, give, 8);
  }
  float y = (up4 ? x[1] : x[0]) + __shfl_xor_sync(ALL, up4 ? x[0] : x[1], 4);
  y *= inv_d;
  y += __shfl_xor_sync(ALL, y, 2);
  y += __shfl_xor_sync(ALL, y, 1);
  if ((lane & 3) == 0) mine[(threadIdx.x >> 5) * 8 + (lane >> 2)] = y;
  __syncthreads();
  // lane l adds value l / 4 of warps l % 4, l % 4 + 4, ...
  float s = 0.0f;
  for (int r = lane & 3; r < (int)(blockDim.x >> 5); r += 4) s += mine[r * 8 + (lane >> 2)];
  s += __shfl_xor_sync(ALL, s, 2);
  s += __shfl_xor_sync(ALL, s, 1);
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(ALL, s, 4 * (i < 3 ? i : i + 1));
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

// A thread's part of a row into a ring stage that holds the row as memory does: of bf16 the
// 16 bytes of vector c, which with split columns other lanes of the warp read; of FP32 its
// own columns.
__device__ __forceinline__ void cp_row(uint4* st, int c, Cols, const __nv_bfloat16* row) {
  cp16(st + c, row + c * NV);
}
__device__ __forceinline__ void cp_row(uint4* st, int, Cols o, const float* row) {
  cp16(st + o.a / 4, row + o.a);
  cp16(st + o.b / 4, row + o.b);
}
template <typename T, bool SPLIT>
__device__ __forceinline__ F8 rd_row(const uint4* st, Cols o) {
  return ld8<SPLIT>(reinterpret_cast<const T*>(st), o);
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
                                          Cols c) {
  F8 f = splat(beta);
  if (w_post) {
    const F8 w = ld8(w_post, c);
#pragma unroll
    for (int j = 0; j < NV / 2; ++j) f.v[j] = mul2(f.v[j], w.v[j]);
  }
  if (gate) {
    const F8 g = ld8(gate, c);
#pragma unroll
    for (int j = 0; j < NV / 2; ++j) f.v[j] = mul2(f.v[j], g.v[j]);
  }
  return f;
}

// FULL: every thread has V vectors of the row.
template <typename RT, int V, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) block_norm_kernel(const FwdK a) {
  constexpr bool KEEP = V <= 2;  // the weights in registers; else read again every row
  constexpr int R = sizeof(RT) / 2, H = NV / 2;
  constexpr bool SPLIT = R == 2;
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) float sh[2 * MAX_WARPS];
  behind();
  int half = 0;
  const int nvec = a.d / NV, tid = threadIdx.x, nt = blockDim.x;
  const int64_t t0 = blockIdx.x * a.rows, t1 = min(t0 + a.rows, a.T);
  const int S = a.stages, row_v = (1 + R) * nvec;  // a stage: y, then res
  if (tid < 2 * MAX_WARPS) sh[tid] = 0.0f;
  __syncthreads();
  auto on = [&](int i) { return FULL || tid + i * nt < nvec; };
  Cols at[V];
#pragma unroll
  for (int i = 0; i < V; ++i) at[i] = cols_of<SPLIT>(tid + i * nt, nvec);
  // the next row to copy, and the row being worked on
  const __nv_bfloat16* y_next = a.y + t0 * a.d;
  const RT* res_next = reinterpret_cast<const RT*>(a.res) + t0 * a.d;
  RT* u_out = reinterpret_cast<RT*>(a.u) + t0 * a.d;
  __nv_bfloat16* n_out = a.n + t0 * a.d;
  int put = 0, get = 0;  // ring stages of those rows
  int left = (int)(t1 - t0);
  auto issue = [&]() {
    if (left > 0) {
      uint4* st = ring + put * row_v;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on(i)) {
          if (a.y) cp_row(st, tid + i * nt, at[i], y_next);
          cp_row(st + nvec, tid + i * nt, at[i], res_next);
        }
      y_next += a.d;
      res_next += a.d;
      --left;
      put = put + 1 == S ? 0 : put + 1;
    }
    cp_commit();
  };
  for (int s = 0; s + 1 < S; ++s) issue();
  F8 f[KEEP ? V : 1], wp[KEEP ? V : 1];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (a.w_pre && on(i)) wp[i] = ld8(a.w_pre, at[i]);
  }
  const float inv_d = 1.0f / a.d;
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
          if (a.y && on(i)) f[i] = post_factor(a.w_post, gate, a.beta, at[i]);
      }
    }
    if (S == 1) {
      __syncthreads();
      issue();
    }
    cp_wait(S > 1 ? S - 2 : 0);
    if (SPLIT) __syncwarp();  // the warp's bf16 rows are in
    const uint4* st = ring + get * row_v;
    get = get + 1 == S ? 0 : get + 1;
    F8 u[V];
    f32x2 s = both(0.0f);
    if (a.y) {
      F8 y[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on(i)) {
          y[i] = rd_row<__nv_bfloat16, SPLIT>(st, at[i]);
#pragma unroll
          for (int j = 0; j < H; ++j) s = fma2(y[i].v[j], y[i].v[j], s);
        }
      float r1 = 1.0f;
      if (a.w_post) r1 = rsqrtf(block_sum1(sum2(s) * inv_d, sh, half) + a.eps);
      const f32x2 rr = both(r1), al = both(a.alpha);
      s = both(0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on(i)) {
          u[i] = rd_row<RT, SPLIT>(st + nvec, at[i]);
          const F8 g = KEEP ? f[KEEP ? i : 0] : post_factor(a.w_post, gate, a.beta, at[i]);
#pragma unroll
          for (int j = 0; j < H; ++j) {
            u[i].v[j] = fma2(al, u[i].v[j], mul2(mul2(g.v[j], rr), y[i].v[j]));
            s = fma2(u[i].v[j], u[i].v[j], s);
          }
          st8<SPLIT>(u_out, at[i], u[i]);
        }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on(i)) {
          u[i] = rd_row<RT, SPLIT>(st + nvec, at[i]);
#pragma unroll
          for (int j = 0; j < H; ++j) s = fma2(u[i].v[j], u[i].v[j], s);
        }
    }
    // a copy refills the stage of the row before this one: every thread has passed a
    // barrier since it read that
    if (a.n) {
      const float ss = block_sum1(sum2(s) * inv_d, sh, half);
      if (S > 1) issue();
      const f32x2 r2 = both(rsqrtf(ss + a.eps));
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on(i)) {
          F8 w = KEEP ? wp[KEEP ? i : 0] : ld8(a.w_pre, at[i]);
#pragma unroll
          for (int j = 0; j < H; ++j) w.v[j] = mul2(mul2(w.v[j], r2), u[i].v[j]);
          st8<SPLIT>(n_out, at[i], w);
        }
    } else {
      if (!a.w_post) __syncthreads();  // as a statistic's barrier
      if (S > 1) issue();
    }
    u_out += a.d;
    n_out += a.d;
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

template <typename RT, int V, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) block_norm_bwd_kernel(const BwdK a) {
  constexpr bool KEEP = V <= 2;
  constexpr int R = sizeof(RT) / 2, H = NV / 2;
  constexpr bool SPLIT = R == 2;
  extern __shared__ uint4 ring[];
  __shared__ float sh[2 * MAX_WARPS * 8];
  behind();
  int half = 0;
  const int nvec = a.d / NV, tid = threadIdx.x, nt = blockDim.x;
  const int64_t t0 = blockIdx.x * a.rows, t1 = min(t0 + a.rows, a.T);
  const int S = a.stages, row_v = (2 + 2 * R) * nvec;  // a stage: dn, y, dres_out, u
  auto on = [&](int i) { return FULL || tid + i * nt < nvec; };
  Cols at[V];
#pragma unroll
  for (int i = 0; i < V; ++i) at[i] = cols_of<SPLIT>(tid + i * nt, nvec);
  // the next row to copy, and the row being worked on
  const int64_t first = t0 * a.d;
  const __nv_bfloat16 *dn_next = a.dn + first, *y_next = a.y + first;
  const RT* du_next = reinterpret_cast<const RT*>(a.du) + first;
  const RT* u_next = reinterpret_cast<const RT*>(a.u) + first;
  RT* dres_out = reinterpret_cast<RT*>(a.dres) + first;
  __nv_bfloat16* dy_out = a.dy + first;
  int put = 0, get = 0;
  int left = (int)(t1 - t0);
  auto issue = [&]() {
    if (left > 0) {
      uint4* st = ring + put * row_v;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on(i)) {
          const int c = tid + i * nt;
          if (a.dn) {
            cp_row(st, c, at[i], dn_next);
            cp_row(st + (2 + R) * nvec, c, at[i], u_next);
          }
          if (a.y) cp_row(st + nvec, c, at[i], y_next);
          if (a.du) cp_row(st + 2 * nvec, c, at[i], du_next);
        }
      dn_next += a.d;
      y_next += a.d;
      du_next += a.d;
      u_next += a.d;
      --left;
      put = put + 1 == S ? 0 : put + 1;
    }
    cp_commit();
  };
  // matrices that are not there read as zeros: no copy ever writes their part of the ring
  if (!a.dn || !a.y || !a.du) {
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on(i)) {
          uint4* st = ring + s * row_v + tid + i * nt;
          const uint4 z = make_uint4(0, 0, 0, 0);
          if (!a.dn) st[0] = z;
          if (!a.y) st[nvec] = z;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (!a.du) st[(2 + r) * nvec] = z;
            if (!a.dn) st[(2 + R + r) * nvec] = z;
          }
        }
    __syncthreads();  // other threads read them
  }
  for (int s = 0; s + 1 < S; ++s) issue();
  F8 sa[V], sb[V], f[KEEP ? V : 1], wp[KEEP ? V : 1];
  const F8 zero = splat(0.0f);
#pragma unroll
  for (int i = 0; i < V; ++i) sa[i] = sb[i] = zero;
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      wp[i] = a.dn && on(i) ? ld8(a.w_pre, at[i]) : zero;
  }
  const float inv_d = 1.0f / a.d;
  const f32x2 alpha = both(a.y ? a.alpha : 1.0f);
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
          f[i] = a.y && on(i) ? post_factor(a.w_post, gate, a.beta, at[i]) : zero;
      }
    }
    if (S == 1) {
      __syncthreads();
      issue();
    }
    cp_wait(S > 1 ? S - 2 : 0);
    if (SPLIT) __syncwarp();  // the warp's bf16 rows are in
    const uint4* st = ring + get * row_v;
    get = get + 1 == S ? 0 : get + 1;
    F8 dn[V], y[V], du[V], u[V];
    auto read = [&](int i) {
      dn[i] = rd_row<__nv_bfloat16, SPLIT>(st, at[i]);
      y[i] = rd_row<__nv_bfloat16, SPLIT>(st + nvec, at[i]);
      du[i] = rd_row<RT, SPLIT>(st + 2 * nvec, at[i]);
      u[i] = rd_row<RT, SPLIT>(st + (2 + R) * nvec, at[i]);
    };
    auto factors = [&](int i, F8& g, F8& w) {
      if constexpr (KEEP) {
        g = f[i];
        w = wp[i];
      } else {
        g = a.y ? post_factor(a.w_post, gate, a.beta, at[i]) : zero;
        w = a.dn ? ld8(a.w_pre, at[i]) : zero;
      }
    };
    f32x2 s[6];
#pragma unroll
    for (int j = 0; j < 6; ++j) s[j] = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (on(i)) {
        read(i);
        F8 g, w;
        factors(i, g, w);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const f32x2 an = mul2(dn[i].v[j], w.v[j]), qy = mul2(g.v[j], y[i].v[j]);
          s[0] = fma2(u[i].v[j], u[i].v[j], s[0]);
          s[1] = fma2(an, u[i].v[j], s[1]);
          s[2] = fma2(y[i].v[j], y[i].v[j], s[2]);
          s[3] = fma2(qy, du[i].v[j], s[3]);
          s[4] = fma2(qy, an, s[4]);
          s[5] = fma2(qy, u[i].v[j], s[5]);
        }
      }
    float sum[6];
#pragma unroll
    for (int j = 0; j < 6; ++j) sum[j] = sum2(s[j]);
    block_mean6(sum, inv_d, sh, half);
    // the stage of the row before this one: every thread has passed a barrier since it read it
    if (S > 1) issue();
    const float r2 = a.dn ? rsqrtf(sum[0] + a.eps) : 0.0f;
    const float r1 = a.w_post ? rsqrtf(sum[2] + a.eps) : 1.0f;
    // the means of a uh and of g v yh
    const float m2 = r2 * sum[1];
    const float m1 =
        a.w_post ? r1 * fmaf(r2, fmaf(-m2, r2 * sum[5], sum[4]), sum[3]) : 0.0f;
    const f32x2 r1p = both(r1), r2p = both(r2), m1n = both(-m1), m2n = both(-m2);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (on(i)) {
        read(i);
        F8 g, w, dres, dy;
        factors(i, g, w);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const f32x2 uh = mul2(u[i].v[j], r2p), yh = mul2(y[i].v[j], r1p);
          const f32x2 v = fma2(r2p, fma2(m2n, uh, mul2(dn[i].v[j], w.v[j])), du[i].v[j]);
          dres.v[j] = mul2(alpha, v);
          dy.v[j] = mul2(r1p, fma2(m1n, yh, mul2(g.v[j], v)));
          sa[i].v[j] = fma2(v, yh, sa[i].v[j]);
          sb[i].v[j] = fma2(dn[i].v[j], uh, sb[i].v[j]);
        }
        st8<SPLIT>(dres_out, at[i], dres);
        if (a.y) st8<SPLIT>(dy_out, at[i], dy);
      }
    dres_out += a.d;
    dy_out += a.d;
    if (t + 1 == t1 || t + 1 == seq_end) {  // the gate row's sums are complete here
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (on(i)) {
          if (a.seq) st8(a.seq + ((int64_t)blockIdx.x + seq) * a.d, at[i], sa[i]);
          if (a.post) {
            float* p = a.post + (int64_t)blockIdx.x * a.d;
            F8 v = flushed ? ld8(p, at[i]) : zero;
            const F8 g = gate ? ld8(gate, at[i]) : splat(1.0f);
#pragma unroll
            for (int j = 0; j < H; ++j) v.v[j] = fma2(g.v[j], sa[i].v[j], v.v[j]);
            st8(p, at[i], v);
          }
          sa[i] = zero;
        }
      flushed = true;
    }
  }
  if (a.pre)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (on(i)) st8(a.pre + (int64_t)blockIdx.x * a.d, at[i], sb[i]);
}

struct FinK {
  const float *post, *pre, *seq, *w_post;
  float *dw_post, *dw_pre, *dgate;
  int64_t T, rows, seq_len;
  int ctas, d, accumulate;
  float beta;
};

// Column sums of the CTAs' rows: job 0 dw_post, 1 dw_pre, 2 + s dgate row s.  A CTA takes
// 32 columns (d is a multiple of 64), four a thread, and as many strands of rows as fit its
// threads, which are added in a fixed order.  Bound by latency: 256 threads have some nine
// rows a strand of the up to 296 CTAs of rows over 2048 columns, all on their way at once;
// narrower rows have up to 2368 CTAs and take 1024 threads.
constexpr int FIN_MOST = 1024;
__global__ void __launch_bounds__(FIN_MOST) block_norm_bwd_finish(const FinK a) {
  __shared__ float4 sh[FIN_MOST / 32][8];
  behind();
  const int x = threadIdx.x & 7, strand = threadIdx.x >> 3, strands = blockDim.x / 8;
  const int cols = a.d / 32;
  const int64_t job = blockIdx.x / cols;
  const int c = (int)(blockIdx.x - job * cols) * 32 + x * 4;
  const float* src;
  float* dst;
  int64_t r0 = 0, r1 = a.ctas;
  float4 f = make_float4(a.beta, a.beta, a.beta, a.beta);
  if (job == 0) {
    src = a.post;
    dst = a.dw_post;
  } else if (job == 1) {
    src = a.pre;
    dst = a.dw_pre;
    f = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  } else {
    const int64_t s = job - 2;
    const int64_t last = min((s + 1) * a.seq_len, a.T) - 1;
    r0 = s * a.seq_len / a.rows + s;
    r1 = last / a.rows + s + 1;
    src = a.seq;
    dst = a.dgate ? a.dgate + s * a.d : nullptr;
    if (a.w_post) {
      const float4 w = *reinterpret_cast<const float4*>(a.w_post + c);
      f = make_float4(f.x * w.x, f.y * w.y, f.z * w.z, f.w * w.w);
    }
  }
  if (dst == nullptr) return;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [](float4& p, const float4& q) {
    p.x += q.x;
    p.y += q.y;
    p.z += q.z;
    p.w += q.w;
  };
  src += c;
#pragma unroll 10
  for (int64_t r = r0 + strand; r < r1; r += strands)
    add(v, *reinterpret_cast<const float4*>(src + r * a.d));
#pragma unroll
  for (int o = 8; o < 32; o <<= 1)
    add(v, make_float4(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o),
                       __shfl_xor_sync(0xffffffffu, v.z, o), __shfl_xor_sync(0xffffffffu, v.w, o)));
  if ((strand & 3) == 0) sh[strand >> 2][x] = v;
  __syncthreads();
  if (strand == 0) {
    for (int i = 1; i < strands / 4; ++i) add(v, sh[i][x]);
    float4* p = reinterpret_cast<float4*>(dst + c);
    float4 o = make_float4(f.x * v.x, f.y * v.y, f.z * v.z, f.w * v.w);
    if (a.accumulate) add(o, *p);
    *p = o;
  }
}

int64_t gate_rows(const moe_dims& dm, const moe_norm_cfg& c) {
  return c.seq_len && dm.T ? (dm.T - 1) / c.seq_len + 1 : 1;
}

// CTAs of a launch over T rows and the rows each takes.
int64_t split_rows(int64_t T, int d, bool bwd, int64_t* rows) {
  const int64_t most = (int64_t)NB_SMS * shape_of(T, d, bwd).per_sm;
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
                const Shape& s, int64_t ctas, cudaStream_t st) {
  const int64_t stage = (int64_t)pieces * (k.d / NV) * 16;
  int64_t n = (NB_SMEM / s.per_sm - 1536) / stage;  // 1 KB a CTA and the static part beside it
  if (n > NB_STAGES) n = NB_STAGES;
  if (n > k.rows + 1) n = k.rows + 1;
  if (n < 1) n = 1;
  k.stages = (int)n;
  const int bytes = (int)(n * stage);
  if (!opt_in(kernel, ready)) return MOE_ERR_CUDA;
  return launch_behind(kernel, ctas, s.threads, bytes, st, k);
}

template <typename RT>
int fwd(const FwdK& k, int64_t ctas, cudaStream_t st) {
  static std::atomic<uint64_t> ready[7];
  const Shape s = shape_of(k.T, k.d, false);
  const int p = 1 + sizeof(RT) / 2;
  const bool full = s.v * s.threads == k.d / NV;
  if (s.v == 1)
    return full ? launch_rows(block_norm_kernel<RT, 1, 256, true>, ready[0], k, p, s, ctas, st)
                : launch_rows(block_norm_kernel<RT, 1, 256, false>, ready[1], k, p, s, ctas, st);
  if (s.v == 2 && s.threads <= 256)
    return full ? launch_rows(block_norm_kernel<RT, 2, 256, true>, ready[2], k, p, s, ctas, st)
                : launch_rows(block_norm_kernel<RT, 2, 256, false>, ready[3], k, p, s, ctas, st);
  if (s.v == 2)
    return full ? launch_rows(block_norm_kernel<RT, 2, 512, true>, ready[4], k, p, s, ctas, st)
                : launch_rows(block_norm_kernel<RT, 2, 512, false>, ready[5], k, p, s, ctas, st);
  return launch_rows(block_norm_kernel<RT, 4, 512, false>, ready[6], k, p, s, ctas, st);
}

template <typename RT>
int bwd(const BwdK& k, int64_t ctas, cudaStream_t st) {
  static std::atomic<uint64_t> ready[7];
  const Shape s = shape_of(k.T, k.d, true);
  const int p = 2 + 2 * (sizeof(RT) / 2);
  const bool full = s.v * s.threads == k.d / NV;
  if (s.v == 1)
    return full ? launch_rows(block_norm_bwd_kernel<RT, 1, 256, true>, ready[0], k, p, s, ctas, st)
                : launch_rows(block_norm_bwd_kernel<RT, 1, 256, false>, ready[1], k, p, s, ctas, st);
  if (s.v == 2 && s.threads <= 256)
    return full ? launch_rows(block_norm_bwd_kernel<RT, 2, 256, true>, ready[2], k, p, s, ctas, st)
                : launch_rows(block_norm_bwd_kernel<RT, 2, 256, false>, ready[3], k, p, s, ctas, st);
  if (s.v == 2)
    return full ? launch_rows(block_norm_bwd_kernel<RT, 2, 512, true>, ready[4], k, p, s, ctas, st)
                : launch_rows(block_norm_bwd_kernel<RT, 2, 512, false>, ready[5], k, p, s, ctas, st);
  return launch_rows(block_norm_bwd_kernel<RT, 4, 512, false>, ready[6], k, p, s, ctas, st);
}

}  // namespace

// For the most CTAs that T tokens or fewer can have, so that the size grows with T (the CTAs
// of a call do not: 296 of one row each for 296 rows of 4096 columns, 150 for 300).
size_t norm_ws_bytes(const moe_dims& dm, const moe_norm_cfg& c) {
  int64_t ctas = 0;
  for (int64_t T : {dm.T, std::min<int64_t>(dm.T, 1)})
    ctas = std::max(ctas, std::min<int64_t>(dm.T, NB_SMS * shape_of(T, dm.d, true).per_sm));
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
  const int64_t ctas = split_rows(dm.T, dm.d, false, &k.rows);
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
  if ((2 + seqs) * (dm.d / 32) >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
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
  const int64_t ctas = split_rows(dm.T, dm.d, true, &k.rows);
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
  return launch_behind(block_norm_bwd_finish, (2 + seqs) * (dm.d / 32), ctas > 320 ? FIN_MOST : 256,
                       0, st, f);
}

}  // namespace moe
