// dact.cuh -- from the gradient of a fused layer's output to the gradient of
// its pre-activation Z, the operand of the input gradient's product, and the
// bias's gradient.
//
//   act:    dZ[m][n]      = dY[m][n] act'(Z[m][n])
//   gated:  dZ[m][2j]     = dY[m][j] Z[m][2j + 1] act'(Z[m][2j])
//           dZ[m][2j + 1] = dY[m][j] act(Z[m][2j])
//   dbias_n = sum_m dZ[m][n]
//
// The product runs on the fp16 tensor cores, so dZ is rounded to fp16 once, or
// carried as two fp16 terms where the product has rows to spare (dx_pair.cuh).
// It is written as dZ m_n 2^(e_m) (dx_pair.cuh: m_n the mantissa of the
// channel scale): the power of two of each row puts the largest |dZ| the row
// can hold near 2^14, so neither a large gradient times a large up value
// overflows nor a small one loses digits, whatever the scale of the loss; the
// product undoes it in fp32.  The bias's gradient sums the fp32 dZ.
#pragma once

#include <math.h>

#include <type_traits>

#include "dx_pair.cuh"
#include "norm.cuh"

namespace qlin {

struct DactArgs {
  const uint16_t* dY;   // [M][N], gated: [M][N / 2]
  const uint16_t* Z;    // [M][N], or null when act is kActNone (never read then)
  const float* cscale;  // c_n [N]
  uint16_t* dZ;         // [M][N] scaled; two terms: [2 M][N], what a row's rounding left in the row behind it
  float* rowscale;      // [M] 2^-e_m
  float* part;          // [G][N] partial column sums (columns kernel)
  float cmul;           // c'_n / c_n
  int M, N, act, G;
  int two;              // dZ in two terms
  int stages;           // ring kernel
};

// dZ of 8 channels in fp32 pairs from their packed values: z (8 halves) and
// dy (8, gated: 4 in x and y).  LIMITS as in act_slopes.
template <bool GATED, bool LIMITS>
__device__ __forceinline__ void dact_vec(int act, const uint4 zv, const uint4 yv, f32x2 (&d)[4]) {
  f32x2 z[4];
  h8_to_f2(zv, z);
  if (GATED) {
    const float2 a = f2_unpack(z[0]), b = f2_unpack(z[1]), c = f2_unpack(z[2]), e = f2_unpack(z[3]);
    const f32x2 gate[2] = {f2_pack(a.x, b.x), f2_pack(c.x, e.x)};
    const f32x2 up[2] = {f2_pack(a.y, b.y), f2_pack(c.y, e.y)};
    const float2 y0 = __half22float2(u32_as_h2(yv.x)), y1 = __half22float2(u32_as_h2(yv.y));
    const f32x2 dy[2] = {f2_pack(y0.x, y0.y), f2_pack(y1.x, y1.y)};
    f32x2 val[2], slope[2];
    act_slopes<LIMITS>(act, gate, val, slope);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 dg = f2_unpack(f2_mul(f2_mul(dy[i], up[i]), slope[i])), du = f2_unpack(f2_mul(dy[i], val[i]));
      d[2 * i] = f2_pack(dg.x, du.x);
      d[2 * i + 1] = f2_pack(dg.y, du.y);
    }
  } else {
    h8_to_f2(yv, d);
    if (act != kActNone) {
      f32x2 val[4], slope[4];
      act_slopes<LIMITS>(act, z, val, slope);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = f2_mul(d[i], slope[i]);
    }
  }
}

// dZ m_n 2^e of the channels of vector v of row m, written in one fp16 term or
// in two (the second is the rest that the first left, rounded).
__device__ __forceinline__ void dact_store(const DactArgs& g, size_t m, int v, const f32x2 (&d)[4], float scale,
                                           const f32x2 (&mant)[4]) {
  f32x2 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f2_mul(f2_mul(d[i], f2_both(scale)), mant[i]);
  const uint4 hi = f2_to_h8(o);
  uint16_t* row = g.dZ + (g.two ? 2 * m : m) * g.N;
  reinterpret_cast<uint4*>(row)[v] = hi;
  if (g.two) {
    f32x2 h[4];
    h8_to_f2(hi, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f2_fma(h[i], f2_both(-1.f), o[i]);
    reinterpret_cast<uint4*>(row + g.N)[v] = f2_to_h8(o);
  }
}
__device__ __forceinline__ void load_mant(const DactArgs& g, int v, f32x2 (&m)[4]) {
  float c[8];
  load_f8(g.cscale + 8 * v, c);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m[i] = f2_pack(chan_mant(__fmul_rn(c[2 * i], g.cmul)), chan_mant(__fmul_rn(c[2 * i + 1], g.cmul)));
}

// The same where chan_mant_is_fraction holds (a power of two in cmul changes
// no fraction): one logic operation a value.
__device__ __forceinline__ float fraction(float c) {
  return __uint_as_float((__float_as_uint(c) & 0x007FFFFFu) | 0x3F800000u);
}
__device__ __forceinline__ void load_fraction(const DactArgs& g, int v, f32x2 (&m)[4]) {
  float c[8];
  load_f8(g.cscale + 8 * v, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = f2_pack(fraction(c[2 * i]), fraction(c[2 * i + 1]));
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN where either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A bound on |dZ| of those channels, up to the factor 1.13 of the slopes
// (and |act(z)| <= |z|).  Gated, an infinity in Z makes it infinite, or NaN
// beside a zero dY (max_nan keeps that); with LIMITS an infinite gate or up
// value counts as 65504.
template <bool GATED, bool LIMITS>
__device__ __forceinline__ float dact_bound(const uint4 zv, const uint4 yv) {
  if (GATED) {
    const uint32_t zw[4] = {zv.x, zv.y, zv.z, zv.w};
    const float2 a = __half22float2(u32_as_h2(yv.x)), b = __half22float2(u32_as_h2(yv.y));
    const float dy[4] = {a.x, a.y, b.x, b.y};
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __habs2(u32_as_h2(zw[i]));
      const float z = __half2float(__hmax(__low2half(h), __high2half(h)));
      top = LIMITS ? fmaxf(top, fabsf(dy[i]) * fminf(z, 65504.f)) : max_nan(top, fabsf(dy[i]) * z);
    }
    return top;
  }
  const __half2 m = __hmax2(__hmax2(__habs2(u32_as_h2(yv.x)), __habs2(u32_as_h2(yv.y))),
                            __hmax2(__habs2(u32_as_h2(yv.z)), __habs2(u32_as_h2(yv.w))));
  return fmaxf(__low2float(m), __high2float(m));
}

// The largest bound of the CTA's threads over nw warps (`red` holds one value
// a warp and is free again after the next barrier); NaN if one is.
__device__ __forceinline__ float dact_top(float top, float* red, int nw) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
  top = lane < nw ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

// 2^e with top 2^e in [2^13, 2^14), as its biased exponent: |dZ m_n| 2^e
// stays below 2^14 * 1.13 * 2.3.  A row of zeros, or one whose dY holds an
// infinity, keeps e = 0.
__device__ __forceinline__ uint32_t dact_exponent(float top) {
  const uint32_t b = __float_as_uint(top) >> 23;
  const uint32_t e = (b == 0u || b == 255u) ? 127u : 267u - b;
  return e > 253u ? 253u : e;
}

// The packed values of vector v of row m from global memory.
template <bool GATED>
__device__ __forceinline__ void dact_load(const DactArgs& g, size_t m, int v, uint4& z, uint4& y) {
  z = make_uint4(0u, 0u, 0u, 0u);
  if (GATED || g.act != kActNone) z = __ldg(reinterpret_cast<const uint4*>(g.Z + m * g.N) + v);
  if (GATED) {
    const uint2 h = __ldg(reinterpret_cast<const uint2*>(g.dY + m * (g.N >> 1)) + v);
    y = make_uint4(h.x, h.y, 0u, 0u);
  } else {
    y = __ldg(reinterpret_cast<const uint4*>(g.dY + m * g.N) + v);
  }
}

constexpr int kDactThreads = 512;
constexpr int kDactRingThreads = 768;  // at most: 80 registers a thread

// One CTA per token row: the row's scale from the bound, then dZ in one more
// pass over the row.
template <bool GATED>
__global__ void __launch_bounds__(kDactThreads) dact_rows_kernel(const __grid_constant__ DactArgs g) {
  __shared__ float red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const size_t m = blockIdx.x;
  const int nv = g.N >> 3;
  auto row = [&](auto lim, float* shared) {  // false: infinities that are still to be limited
    constexpr bool kLimits = decltype(lim)::value;
    float top = 0.f;
    for (int v = threadIdx.x; v < nv; v += kDactThreads) {
      uint4 z, y;
      dact_load<GATED>(g, m, v, z, y);
      top = max_nan(top, dact_bound<GATED, kLimits>(z, y));
    }
    top = dact_top(top, shared, kDactThreads / 32);
    if (!kLimits && !(top < INFINITY)) return false;
    const uint32_t e = dact_exponent(top);
    const float scale = __uint_as_float(e << 23);
    if (threadIdx.x == 0) g.rowscale[m] = __uint_as_float((254u - e) << 23);
    for (int v = threadIdx.x; v < nv; v += kDactThreads) {
      uint4 z, y;
      f32x2 d[4], c[4];
      dact_load<GATED>(g, m, v, z, y);
      dact_vec<GATED, kLimits>(g.act, z, y, d);
      load_mant(g, v, c);
      dact_store(g, m, v, d, scale, c);
    }
    return true;
  };
  // (not gated: the bound does not see Z)
  if (!GATED || !row(std::false_type{}, red[0])) row(std::true_type{}, red[1]);
}

// Partial column sums of dZ: thread t of CTA (x, y) owns the 8 channels of
// vector 128 x + t and the rows y, y + G, ...
template <bool GATED>
__global__ void __launch_bounds__(128) dact_columns_kernel(const __grid_constant__ DactArgs g) {
  griddep_launch_dependents();
  griddep_wait();
  const int v = blockIdx.x * 128 + threadIdx.x;
  if (v >= (g.N >> 3)) return;
  f32x2 s[4] = {f2_both(0.f), f2_both(0.f), f2_both(0.f), f2_both(0.f)};
#pragma unroll 2
  for (int m = blockIdx.y; m < g.M; m += g.G) {
    uint4 z, y;
    f32x2 d[4];
    dact_load<GATED>(g, m, v, z, y);
    dact_vec<GATED, true>(g.act, z, y, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = f2_add(s[i], d[i]);
  }
  store_f2x4(g.part + static_cast<size_t>(blockIdx.y) * g.N + 8 * v, s);
}

// Both at once over a row ring (norm.cuh, one row a stage): persistent CTAs of
// T threads, the next rows on their way by bulk copies, thread t owning the
// vectors t, t + T, ... (VPT at most).  One barrier a row, for the maximum of the bound;
// the mantissas of the channel factors stay in registers where they fit
// beside the column sums, which ACC keeps over the CTA's rows and writes once
// as partial row blockIdx.x.  dZ is skipped when it is null (only the bias's
// gradient is wanted).  2048 x 11008, GELU (tanh), 38 us = 3.6 TB/s; gated 2048 x
// 22016, SiLU, 47 us = 4.8 TB/s.  Nothing is saturated (first case: issue slots
// half used, DRAM a third): with one CTA of 22 warps an SM, what a warp waits
// for is spread over dependent arithmetic, shared memory and the special
// functions, the row's barrier (an eighth) and the next row.  Two rows at a time
// gave nothing, nor did two CTAs of half the threads (41 us).
template <bool GATED, int VPT, bool ACC>
__global__ void __launch_bounds__(kDactRingThreads) dact_ring_kernel(const __grid_constant__ DactArgs g) {
  constexpr bool kKeep = VPT * (ACC ? 2 : 1) <= 4;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ float red[3][32];
  __shared__ uint64_t full[kRingStages];
  __shared__ int abort_flag;
  const int t = threadIdx.x, T = static_cast<int>(blockDim.x), nw = T >> 5;
  const int nv = g.N >> 3;
  const bool has_z = GATED || g.act != kActNone;
  const uint32_t zb = has_z ? static_cast<uint32_t>(g.N) * 2u : 0u;  // bytes of a row
  const uint32_t yb = static_cast<uint32_t>(g.N) * (GATED ? 1u : 2u);
  const size_t stage = zb + yb;
  const int S = g.stages;
  if (t == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  const size_t step = gridDim.x, M = static_cast<size_t>(g.M);
  int issued = 0;  // rows on their way (thread 0)
  auto load = [&](size_t m, int s) {
    unsigned char* dst = ring_smem + s * stage;
    mbar_arrive_expect_tx(&full[s], zb + yb);
    if (has_z) bulk_load(dst, g.Z + m * g.N, zb, &full[s]);
    bulk_load(dst + zb, g.dY + m * (GATED ? g.N >> 1 : g.N), yb, &full[s]);
    ++issued;
  };
  if (t == 0)
    for (int s = 0; s < S; ++s)
      if (blockIdx.x + s * step < M) load(blockIdx.x + s * step, s);
  f32x2 sum[ACC ? VPT : 1][4], mant[kKeep ? VPT : 1][4];
  bool inside = true;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (ACC) sum[j][e] = f2_both(0.f);
      if (kKeep) mant[j][e] = f2_both(0.f);
    }
    if (t + j * T < nv) {
      if (kKeep) {
        load_mant(g, t + j * T, mant[kKeep ? j : 0]);
      } else {
        float c[8];
        load_f8(g.cscale + 8 * (t + j * T), c);
#pragma unroll
        for (int e = 0; e < 8; ++e) inside = inside && chan_mant_is_fraction(__fmul_rn(c[e], g.cmul));
      }
    }
  }
  // the usual case: every channel factor's mantissa is its fraction field
  if (!kKeep) inside = __syncthreads_and(inside);
  bool ok = true;  // a thread whose wait gave up waits no more: what follows it is not used
  int i = 0;
  for (size_t m = blockIdx.x; m < M; m += step, ++i) {
    const int s = i % S;
    if (ok && !mbar_wait(&full[s], static_cast<uint32_t>(i / S) & 1u, &abort_flag)) ok = false;
    const uint4* zr = reinterpret_cast<const uint4*>(ring_smem + s * stage);
    const unsigned char* yr = ring_smem + s * stage + zb;
    auto values = [&](int v, uint4& z, uint4& y) {
      z = has_z ? zr[v] : make_uint4(0u, 0u, 0u, 0u);
      if (GATED) {
        const uint2 h = reinterpret_cast<const uint2*>(yr)[v];
        y = make_uint4(h.x, h.y, 0u, 0u);
      } else {
        y = reinterpret_cast<const uint4*>(yr)[v];
      }
    };
    auto bound = [&](auto lim, float* shared) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (t + j * T < nv) {
          uint4 z, y;
          values(t + j * T, z, y);
          top = max_nan(top, dact_bound<GATED, decltype(lim)::value>(z, y));
        }
      }
      return dact_top(top, shared, nw);
    };
    auto write = [&](auto lim, float top) {
      const uint32_t ex = dact_exponent(top);
      const float scale = __uint_as_float(ex << 23);
      if (t == 0 && g.dZ) g.rowscale[m] = __uint_as_float((254u - ex) << 23);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = t + j * T;
        if (v < nv) {
          uint4 z, y;
          f32x2 d[4];
          values(v, z, y);
          dact_vec<GATED, decltype(lim)::value>(g.act, z, y, d);
          if (ACC) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[j][e] = f2_add(sum[j][e], d[e]);
          }
          if (g.dZ) {
            f32x2 c[4];
            if (!kKeep) {
              if (inside) load_fraction(g, v, c);
              else load_mant(g, v, c);
            }
            dact_store(g, m, v, d, scale, kKeep ? mant[kKeep ? j : 0] : c);
          }
        }
      }
    };
    const float top = bound(std::bool_constant<!GATED>{}, red[i & 1]);
    if (t == 0 && i > 0 && abort_flag == 0) {  // the previous row's stage: every thread is done with it
      const size_t next = m + static_cast<size_t>(S - 1) * step;
      if (next < M) load(next, (i - 1) % S);
    }
    // gated: infinities in the row, or NaN, take the bound again (not gated it does not see Z)
    if (GATED && top < INFINITY) write(std::false_type{}, top);
    else write(std::true_type{}, GATED ? bound(std::true_type{}, red[2]) : top);
  }
  if (t == 0 && abort_flag) drain_ring(full, S, issued);  // no copy outlives the CTA
  if (ACC) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = t + j * T;
      if (v < nv) store_f2x4(g.part + static_cast<size_t>(blockIdx.x) * g.N + 8 * v, sum[j]);
    }
  }
}

}  // namespace qlin
