// norm.cuh -- layer norm and RMS norm in front of the quantized linear
// layer: forward, and backward with the reduction of the weight's and the
// bias's gradients over the tokens.
//
//   mu_m = mean_k x[m][k] (0 for RMS),  r_m = 1 / sqrt(mean_k (x - mu)^2 + eps)
//   xh   = (x - mu_m) r_m,              y = xh gamma_k + beta_k
//   dx   = r_m (w - mean_k w - xh mean_k(w xh)) + dres,  w = dy gamma_k
//          (without the mean_k w term for RMS)
//   dgamma_k = sum_m dy xh,             dbeta_k = sum_m dy
//
// Everything between the fp16 inputs and outputs is fp32: the statistics are
// taken in two passes over the row held on chip (the sum of squares of
// x - mu, not of x, so a large mean costs no digits), and each output is
// rounded once.  Sums are added in an order that depends on the shape alone,
// so results repeat bit for bit.
#pragma once

#include "gemm.cuh"
#include "pack.cuh"

namespace qlin {

struct NormFwdArgs {
  const uint16_t* X;   // [M][K]
  const float* gamma;  // [K]
  const float* beta;   // [K] or null
  uint16_t* Y;         // [M][K]
  float* mean;         // [M] or null
  float* rstd;         // [M] or null
  int M, K, rms;
  float eps;
  int stages;          // ring kernel
};

struct NormBwdArgs {
  const uint16_t* dY;    // [M][K]
  const uint16_t* X;     // [M][K]
  const float* gamma;    // [K]
  const float* mean;     // [M], null for RMS
  const float* rstd;     // [M]
  const uint16_t* dres;  // [M][K] or null
  uint16_t* dX;          // [M][K]
  float* part;           // partial column sums: [G][K] of dgamma, then [G][K] of dbeta; null when none is wanted
  int M, K, rms, G;
  int stages;            // ring kernel
};

__device__ __forceinline__ void h8_to_f(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 h = *reinterpret_cast<const __half2*>(&w[e]);
    const float2 t = __half22float2(h);
    f[2 * e] = t.x;
    f[2 * e + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 f_to_h8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 h = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load_f8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ void load_f2x4(const float* p, f32x2 (&f)[4]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = f2_pack(a.x, a.y);
  f[1] = f2_pack(a.z, a.w);
  f[2] = f2_pack(b.x, b.y);
  f[3] = f2_pack(b.z, b.w);
}
__device__ __forceinline__ void store_f2x4(float* p, const f32x2 (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float2 a = f2_unpack(f[2 * e]), b = f2_unpack(f[2 * e + 1]);
    reinterpret_cast<float4*>(p)[e] = make_float4(a.x, a.y, b.x, b.y);
  }
}
__device__ __forceinline__ float f2_sum(f32x2 v) {
  const float2 t = f2_unpack(v);
  return t.x + t.y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the T threads of a row.  `red` holds T / 32 floats and is free
// again only after the next barrier: callers alternate two of them.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (T == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) s += red[w];
  return s;
}

// Forward, for calls with fewer rows than the ring kernel has CTAs, and for
// rows too long for it: one token of 4096 takes 2.4 us, which is the launch.
// T threads share a row (four rows per CTA when T is one warp);
// thread t holds the 8-element vectors t, t + T, ... of the row in
// registers, VPT of them at most.
template <int T, int VPT>
__global__ void __launch_bounds__(T == 32 ? 128 : T) norm_forward_kernel(const __grid_constant__ NormFwdArgs g) {
  __shared__ float red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int t = T == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int m = T == 32 ? static_cast<int>(blockIdx.x) * 4 + (threadIdx.x >> 5) : static_cast<int>(blockIdx.x);
  if (m >= g.M) return;  // whole warps (T = 32) or nobody
  const int nv = g.K >> 3;
  const uint4* xr = reinterpret_cast<const uint4*>(g.X + static_cast<size_t>(m) * g.K);
  uint4 x[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = t + j * T;
    x[j] = v < nv ? __ldg(xr + v) : make_uint4(0u, 0u, 0u, 0u);
  }
  const float invk = 1.f / static_cast<float>(g.K);
  float mu = 0.f;
  if (!g.rms) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float f[8];
      h8_to_f(x[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += f[e];
    }
    mu = row_sum<T>(s, red[0]) * invk;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (t + j * T < nv) {
      float f[8];
      h8_to_f(x[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(f[e] - mu, f[e] - mu, q);
    }
  }
  const float r = rsqrtf(fmaf(row_sum<T>(q, red[1]), invk, g.eps));
  uint4* yr = reinterpret_cast<uint4*>(g.Y + static_cast<size_t>(m) * g.K);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = t + j * T;
    if (v < nv) {
      float f[8], gm[8], bt[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      h8_to_f(x[j], f);
      load_f8(g.gamma + 8 * v, gm);
      if (g.beta) load_f8(g.beta + 8 * v, bt);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mu) * r, gm[e], bt[e]);
      yr[v] = f_to_h8(f);
    }
  }
  if (t == 0) {
    if (g.mean) g.mean[m] = mu;
    if (g.rstd) g.rstd[m] = r;
  }
}

// Column sums of dy xh and dy over a block of rows: thread t of CTA (x, y)
// owns the 8 columns of vector 128 x + t and the rows y, y + G, ...
__global__ void __launch_bounds__(128) norm_columns_kernel(const __grid_constant__ NormBwdArgs g) {
  griddep_launch_dependents();
  griddep_wait();
  const int v = blockIdx.x * 128 + threadIdx.x;
  if (v >= (g.K >> 3)) return;
  float sg[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sb[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int m = blockIdx.y; m < g.M; m += g.G) {
    const size_t o = static_cast<size_t>(m) * g.K;
    float x[8], dy[8];
    h8_to_f(__ldg(reinterpret_cast<const uint4*>(g.X + o) + v), x);
    h8_to_f(__ldg(reinterpret_cast<const uint4*>(g.dY + o) + v), dy);
    const float mu = g.rms ? 0.f : __ldg(g.mean + m), r = __ldg(g.rstd + m);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sg[e] = fmaf(dy[e], (x[e] - mu) * r, sg[e]);
      sb[e] += dy[e];
    }
  }
  float4* pg = reinterpret_cast<float4*>(g.part + static_cast<size_t>(blockIdx.y) * g.K) + 2 * v;
  float4* pb = reinterpret_cast<float4*>(g.part + static_cast<size_t>(g.G + blockIdx.y) * g.K) + 2 * v;
  pg[0] = make_float4(sg[0], sg[1], sg[2], sg[3]);
  pg[1] = make_float4(sg[4], sg[5], sg[6], sg[7]);
  pb[0] = make_float4(sb[0], sb[1], sb[2], sb[3]);
  pb[1] = make_float4(sb[4], sb[5], sb[6], sb[7]);
}

// out[k] = sum over the G partial rows of part [G][K], in one order: the W
// warps of the CTA take the rows w, w + W, ... of 32 columns, and their sums
// are added in order.
template <int W>
__device__ __forceinline__ void column_sum(const float* __restrict__ part, int G, int K, int block,
                                           float* __restrict__ out) {
  __shared__ float red[W][32];
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int k = block * 32 + c;
  const float* p = part + k;
  float s = 0.f;
  if (k < K) {
#pragma unroll 16
    for (int i = w; i < G; i += W) s += __ldcg(p + static_cast<size_t>(i) * K);
  }
  red[w][c] = s;
  __syncthreads();
  if (w == 0 && k < K) {
#pragma unroll
    for (int i = 1; i < W; ++i) s += red[i][c];
    out[k] = s;
  }
}

// dgamma (blockIdx.y = 0) and dbeta (1) from part [2][G][K]; either may be null.
template <int W>
__global__ void __launch_bounds__(32 * W) column_sum_kernel(const float* __restrict__ part, int G, int K,
                                                          float* __restrict__ out0, float* __restrict__ out1) {
  griddep_launch_dependents();
  griddep_wait();
  float* out = blockIdx.y ? out1 : out0;
  if (out) column_sum<W>(part + static_cast<size_t>(blockIdx.y) * G * K, G, K, static_cast<int>(blockIdx.x), out);
}

// ---- Row rings: persistent CTAs work through groups of R neighbouring rows,
// blockIdx.x, + gridDim.x, ...; one thread keeps the next groups on their way
// into shared memory with bulk copies, so the loads do not wait for the rows
// in hand and need no registers.  Thread t owns the 8-element vectors t,
// t + T, ... of every row, VPT of them at most (T threads a CTA).  A row
// costs its element work and a share of a barrier: R rows reduce together,
// which is what a row at a time spent most of its time on.
constexpr int kRingStages = 3;  // at most; two where that lets more CTAs share an SM

// Sums of NV values over the CTA's `nw` warps, returned to every thread.  In
// the warp, lanes exchange halves of the values (recursive halving), so NV
// values cost about NV + 3 shuffles instead of 5 NV; the warps' sums meet in
// `red` ([NV][32], one of two alternating buffers: one barrier a call).
template <int NV>
__device__ __forceinline__ void cta_sums(float (&v)[NV], float (*red)[32], int nw) {
  static_assert(NV == 1 || NV == 2 || NV == 4 || NV == 8, "a power of two up to 8");
  const int lane = threadIdx.x & 31;
  float x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = v[i];
  // after the step of lane bit b, lanes with the bit set keep the upper half
#pragma unroll
  for (int n = NV / 2, b = 16; n >= 1; n >>= 1, b >>= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? x[i] : x[n + i];
      const float keep = up ? x[n + i] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, b);
    }
  }
#pragma unroll
  for (int b = 16 / NV; b >= 1; b >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], b);
  // lane bits 16, 8, 4 (as many as halvings) name the value held
  constexpr int kSpan = 32 / NV;  // lanes that hold the same value
  const int mine = lane / kSpan;
  if (nw > 1) {
    if (lane % kSpan == 0) red[mine][threadIdx.x >> 5] = x[0];
    __syncthreads();
    x[0] = 0.f;
    for (int w = lane % kSpan; w < nw; w += kSpan) x[0] += red[mine][w];
#pragma unroll
    for (int b = kSpan / 2; b >= 1; b >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], b);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = __shfl_sync(0xffffffffu, x[0], i * kSpan);
}

// A group of rows [row, row + n) of the arrays a, b, c (the last two may be
// null), one array after the other in the stage, R rows apart.
__device__ __forceinline__ void ring_load(unsigned char* dst, const uint16_t* a, const uint16_t* b, const uint16_t* c,
                                          size_t row, int n, int R, int K, uint64_t* bar) {
  const uint32_t bytes = static_cast<uint32_t>(n) * static_cast<uint32_t>(K) * 2u;
  const size_t next = static_cast<size_t>(R) * K * 2;
  mbar_arrive_expect_tx(bar, bytes * (1u + (b ? 1u : 0u) + (c ? 1u : 0u)));
  bulk_load(dst, a + row * K, bytes, bar);
  if (b) bulk_load(dst + next, b + row * K, bytes, bar);
  if (c) bulk_load(dst + 2 * next, c + row * K, bytes, bar);
}

__device__ __forceinline__ int group_rows(size_t grp, int R, int M) {  // rows of group grp that exist
  const size_t left = static_cast<size_t>(M) - grp * R;
  return left < static_cast<size_t>(R) ? static_cast<int>(left) : R;
}

// Forward over a ring.  gamma and beta stay in registers.  8192 x 8192 layer
// norm: 47.8 us, 5.6 TB/s of the row's one read and one write (a copy: 6.5).
template <int VPT, int R>
__global__ void __launch_bounds__(512) norm_forward_ring_kernel(const __grid_constant__ NormFwdArgs g) {
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ float red[4][R][32];
  __shared__ uint64_t full[kRingStages];
  __shared__ int abort_flag;
  const int t = threadIdx.x, T = static_cast<int>(blockDim.x), nw = T >> 5;
  const int nv = g.K >> 3, S = g.stages;
  const size_t stage = static_cast<size_t>(R) * g.K * 2;
  const size_t groups = (static_cast<size_t>(g.M) + R - 1) / R, step = gridDim.x;
  if (t == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  int issued = 0;  // groups on their way (thread 0)
  auto load = [&](size_t grp, int s) {
    ring_load(ring_smem + s * stage, g.X, nullptr, nullptr, grp * R, group_rows(grp, R, g.M), R, g.K, &full[s]);
    ++issued;
  };
  if (t == 0)
    for (int s = 0; s < S; ++s)
      if (blockIdx.x + s * step < groups) load(blockIdx.x + s * step, s);
  f32x2 gm[VPT][4], bt[VPT][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = t + j * T;
#pragma unroll
    for (int e = 0; e < 4; ++e) gm[j][e] = bt[j][e] = f2_both(0.f);
    if (v < nv) {
      load_f2x4(g.gamma + 8 * v, gm[j]);
      if (g.beta) load_f2x4(g.beta + 8 * v, bt[j]);
    }
  }
  const float invk = 1.f / static_cast<float>(g.K);
  bool ok = true;  // a thread whose wait gave up waits no more: what follows it is not used
  int i = 0;
  for (size_t grp = blockIdx.x; grp < groups; grp += step, ++i) {
    const int s = i % S;
    const int rows = group_rows(grp, R, g.M);
    const size_t m0 = grp * R;
    if (ok && !mbar_wait(&full[s], static_cast<uint32_t>(i / S) & 1u, &abort_flag)) ok = false;
    const uint4* xr = reinterpret_cast<const uint4*>(ring_smem + s * stage);
    f32x2 x[R][VPT][4];  // the rows' values, then x - mu
    float mu[R], q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        h8_to_f2(t + j * T < nv ? xr[r * nv + t + j * T] : make_uint4(0u, 0u, 0u, 0u), x[r][j]);
      mu[r] = 0.f;
    }
    if (!g.rms) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        f32x2 a = x[r][0][0];
#pragma unroll
        for (int k = 1; k < 4 * VPT; ++k) a = f2_add(a, x[r][k >> 2][k & 3]);
        mu[r] = f2_sum(a);
      }
      cta_sums<R>(mu, red[2 * (i & 1)], nw);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        mu[r] *= invk;
        const f32x2 nmu = f2_both(-mu[r]);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          if (t + j * T < nv)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[r][j][e] = f2_add(x[r][j][e], nmu);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f32x2 a = f2_mul(x[r][0][0], x[r][0][0]);
#pragma unroll
      for (int k = 1; k < 4 * VPT; ++k) a = f2_fma(x[r][k >> 2][k & 3], x[r][k >> 2][k & 3], a);
      q[r] = f2_sum(a);
    }
    cta_sums<R>(q, red[2 * (i & 1) + 1], nw);
    if (nw == 1) __syncwarp();
    // every thread holds its part of the rows (the sums' barrier): refill
    if (t == 0) {
      const size_t next = grp + static_cast<size_t>(S) * step;
      if (abort_flag == 0 && next < groups) load(next, s);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      const float rs = rsqrtf(fmaf(q[r], invk, g.eps));
      const f32x2 r2 = f2_both(rs);
      uint4* yr = reinterpret_cast<uint4*>(g.Y + (m0 + r) * g.K);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (t + j * T < nv) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[r][j][e] = f2_fma(f2_mul(x[r][j][e], r2), gm[j][e], bt[j][e]);
          yr[t + j * T] = f2_to_h8(x[r][j]);
        }
      }
      if (t == 0) {
        if (g.mean) g.mean[m0 + r] = mu[r];
        if (g.rstd) g.rstd[m0 + r] = rs;
      }
    }
  }
  if (t == 0 && abort_flag) drain_ring(full, S, issued);  // no copy outlives the CTA
}

// Backward over a ring: dX, and with ACC the column sums of dy xh and dy over
// the CTA's rows in registers, written once as partial row blockIdx.x.  The
// two sums of R rows are taken together: one barrier a group.  A stage is
// refilled after the next group's barrier, when every thread is done with
// it; xh and dy gamma are formed again from shared memory rather than kept.
// gamma stays in registers where it fits (VPT <= 2).
// 4099 x 4096 layer norm with dres: 28 us = 4.8 TB/s, 31.7 with the column
// sums' launch.
template <int VPT, int R, bool ACC>
__global__ void __launch_bounds__(512) norm_backward_ring_kernel(const __grid_constant__ NormBwdArgs g) {
  constexpr bool kGamma = VPT <= 2;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ float red[2][2 * R][32];
  __shared__ uint64_t full[kRingStages];
  __shared__ int abort_flag;
  const int t = threadIdx.x, T = static_cast<int>(blockDim.x), nw = T >> 5;
  const int nv = g.K >> 3, S = g.stages;
  const size_t part = static_cast<size_t>(R) * g.K * 2;
  const size_t stage = part * (g.dres ? 3 : 2);
  const size_t groups = (static_cast<size_t>(g.M) + R - 1) / R, step = gridDim.x;
  if (t == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  int issued = 0;  // groups on their way (thread 0)
  auto load = [&](size_t grp, int s) {
    ring_load(ring_smem + s * stage, g.dY, g.X, g.dres, grp * R, group_rows(grp, R, g.M), R, g.K, &full[s]);
    ++issued;
  };
  if (t == 0)
    for (int s = 0; s < S; ++s)
      if (blockIdx.x + s * step < groups) load(blockIdx.x + s * step, s);
  f32x2 sg[VPT][4], sb[VPT][4], gk[kGamma ? VPT : 1][4];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) sg[j][e] = sb[j][e] = f2_both(0.f);
  if (kGamma) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) gk[kGamma ? j : 0][e] = f2_both(0.f);
      if (t + j * T < nv) load_f2x4(g.gamma + 8 * (t + j * T), gk[kGamma ? j : 0]);
    }
  }
  const float invk = 1.f / static_cast<float>(g.K);
  float mu1[R], rs1[R];  // the next group's statistics, on their way a group ahead
  auto statistics = [&](size_t grp) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const size_t m = grp * R + r;
      const bool in = m < static_cast<size_t>(g.M);
      mu1[r] = in && !g.rms ? g.mean[m] : 0.f;
      rs1[r] = in ? g.rstd[m] : 0.f;
    }
  };
  statistics(blockIdx.x);
  bool ok = true;  // a thread whose wait gave up waits no more: what follows it is not used
  int i = 0;
  for (size_t grp = blockIdx.x; grp < groups; grp += step, ++i) {
    const int s = i % S;
    const int rows = group_rows(grp, R, g.M);
    const size_t m0 = grp * R;
    float mu[R], rs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mu[r] = mu1[r];
      rs[r] = rs1[r];
    }
    statistics(grp + step);
    if (ok && !mbar_wait(&full[s], static_cast<uint32_t>(i / S) & 1u, &abort_flag)) ok = false;
    const uint4* dr = reinterpret_cast<const uint4*>(ring_smem + s * stage);
    const uint4* xr = reinterpret_cast<const uint4*>(ring_smem + s * stage + part);
    const uint4* rr = reinterpret_cast<const uint4*>(ring_smem + s * stage + 2 * part);
    float sum[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f32x2 a1 = f2_both(0.f), a2 = f2_both(0.f);
      const f32x2 nmu = f2_both(-mu[r]), r2 = f2_both(rs[r]);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = t + j * T;
        if (v < nv && r < rows) {
          f32x2 xh[4], dy[4], gm[4];
          h8_to_f2(xr[r * nv + v], xh);
          h8_to_f2(dr[r * nv + v], dy);
          if (!kGamma) load_f2x4(g.gamma + 8 * v, gm);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            xh[e] = f2_mul(f2_add(xh[e], nmu), r2);
            if (ACC) {
              sg[j][e] = f2_fma(dy[e], xh[e], sg[j][e]);
              sb[j][e] = f2_add(sb[j][e], dy[e]);
            }
            const f32x2 w = f2_mul(dy[e], kGamma ? gk[kGamma ? j : 0][e] : gm[e]);
            a1 = f2_add(a1, w);
            a2 = f2_fma(w, xh[e], a2);
          }
        }
      }
      sum[2 * r] = f2_sum(a1);
      sum[2 * r + 1] = f2_sum(a2);
    }
    cta_sums<2 * R>(sum, red[i & 1], nw);
    if (nw == 1) __syncwarp();
    if (t == 0 && i > 0 && abort_flag == 0) {  // the previous group's stage
      const size_t next = grp + static_cast<size_t>(S - 1) * step;
      if (next < groups) load(next, (i - 1) % S);
    }
    if (g.dX) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        const f32x2 nmu = f2_both(-mu[r]), r2 = f2_both(rs[r]);
        const f32x2 n1 = f2_both(g.rms ? 0.f : -sum[2 * r] * invk), n2 = f2_both(-sum[2 * r + 1] * invk);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int v = t + j * T;
          if (v < nv) {
            f32x2 x[4], dy[4], gm[4], res[4];
            h8_to_f2(xr[r * nv + v], x);
            h8_to_f2(dr[r * nv + v], dy);
            if (!kGamma) load_f2x4(g.gamma + 8 * v, gm);
            h8_to_f2(g.dres ? rr[r * nv + v] : make_uint4(0u, 0u, 0u, 0u), res);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const f32x2 xh = f2_mul(f2_add(x[e], nmu), r2);
              x[e] = f2_fma(f2_fma(xh, n2, f2_add(f2_mul(dy[e], kGamma ? gk[kGamma ? j : 0][e] : gm[e]), n1)), r2, res[e]);
            }
            reinterpret_cast<uint4*>(g.dX + (m0 + r) * g.K)[v] = f2_to_h8(x);
          }
        }
      }
    }
  }
  if (t == 0 && abort_flag) drain_ring(full, S, issued);  // no copy outlives the CTA
  if (ACC) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = t + j * T;
      if (v < nv) {
        store_f2x4(g.part + static_cast<size_t>(blockIdx.x) * g.K + 8 * v, sg[j]);
        store_f2x4(g.part + (step + blockIdx.x) * g.K + 8 * v, sb[j]);
      }
    }
  }
}

// Input gradient, one CTA of T threads per row, the row read twice (the
// second time from L2).  dX may be the buffer of dY, X or dres: each thread
// writes only the vectors it has just read.
template <int T>
__global__ void __launch_bounds__(T) norm_rows_kernel(const __grid_constant__ NormBwdArgs g) {
  __shared__ float red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int m = static_cast<int>(blockIdx.x);
  const int nv = g.K >> 3;
  const size_t o = static_cast<size_t>(m) * g.K;
  const uint4* xr = reinterpret_cast<const uint4*>(g.X + o);
  const uint4* dr = reinterpret_cast<const uint4*>(g.dY + o);
  const float mu = g.rms ? 0.f : g.mean[m], r = g.rstd[m];
  float s1 = 0.f, s2 = 0.f;
  for (int v = threadIdx.x; v < nv; v += T) {
    float x[8], dy[8], gm[8];
    h8_to_f(xr[v], x);
    h8_to_f(dr[v], dy);
    load_f8(g.gamma + 8 * v, gm);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float w = dy[e] * gm[e];
      s1 += w;
      s2 = fmaf(w, (x[e] - mu) * r, s2);
    }
  }
  const float invk = 1.f / static_cast<float>(g.K);
  s1 = row_sum<T>(s1, red[0]) * invk;
  s2 = row_sum<T>(s2, red[1]) * invk;
  if (g.rms) s1 = 0.f;
  for (int v = threadIdx.x; v < nv; v += T) {
    float x[8], dy[8], gm[8], rs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    h8_to_f(xr[v], x);
    h8_to_f(dr[v], dy);
    load_f8(g.gamma + 8 * v, gm);
    if (g.dres) h8_to_f(reinterpret_cast<const uint4*>(g.dres + o)[v], rs);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float xh = (x[e] - mu) * r;
      x[e] = fmaf(r, dy[e] * gm[e] - s1 - xh * s2, rs[e]);
    }
    reinterpret_cast<uint4*>(g.dX + o)[v] = f_to_h8(x);
  }
}

}  // namespace qlin
