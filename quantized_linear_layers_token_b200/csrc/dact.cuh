// dact.cuh -- from the gradient of a fused layer's output to the gradient of
// its pre-activation Z, the operand of the input gradient's product, and the
// bias's gradient.
//
//   act:    dZ[m][n]      = dY[m][n] act'(Z[m][n])
//   gated:  dZ[m][2j]     = dY[m][j] Z[m][2j + 1] act'(Z[m][2j])
//           dZ[m][2j + 1] = dY[m][j] act(Z[m][2j])
//   dbias_n = sum_m dZ[m][n]
//
// The product runs on the fp16 tensor cores, so dZ is rounded to fp16 once.
// It is written as dZ m_n 2^(e_m) (dx_pair.cuh: m_n the mantissa of the
// channel scale): the power of two of each row puts the largest |dZ| the row
// can hold near 2^14, so neither a large gradient times a large up value
// overflows nor a small one loses digits, whatever the scale of the loss; the
// product undoes it in fp32.  The bias's gradient sums the fp32 dZ.
#pragma once

#include "dx_pair.cuh"
#include "norm.cuh"

namespace qlin {

struct DactArgs {
  const uint16_t* dY;   // [M][N], gated: [M][N / 2]
  const uint16_t* Z;    // [M][N], or null when act is kActNone (never read then)
  const float* cscale;  // c_n [N]
  uint16_t* dZ;         // [M][N] scaled (rows kernel)
  float* rowscale;      // [M] 2^-e_m (rows kernel)
  float* part;          // [G][N] partial column sums (columns kernel)
  float cmul;           // c'_n / c_n
  int M, N, act, G;
};

// dZ of the 8 channels of vector v of row m, in fp32.
template <bool GATED>
__device__ __forceinline__ void dact_vec(const DactArgs& g, size_t m, int v, float (&d)[8]) {
  float z[8];
  if (GATED || g.act != kActNone) h8_to_f(__ldg(reinterpret_cast<const uint4*>(g.Z + m * g.N) + v), z);
  if (GATED) {
    const uint2 h = __ldg(reinterpret_cast<const uint2*>(g.dY + m * (g.N >> 1)) + v);
    const float2 a = __half22float2(u32_as_h2(h.x)), b = __half22float2(u32_as_h2(h.y));
    const float dy[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float val, slope;
      act_slope(g.act, z[2 * i], val, slope);
      d[2 * i] = dy[i] * z[2 * i + 1] * slope;
      d[2 * i + 1] = dy[i] * val;
    }
  } else {
    h8_to_f(__ldg(reinterpret_cast<const uint4*>(g.dY + m * g.N) + v), d);
    if (g.act != kActNone) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float val, slope;
        act_slope(g.act, z[i], val, slope);
        d[i] *= slope;
      }
    }
  }
}

constexpr int kDactThreads = 512;

// One CTA per token row: the row's scale from a bound on |dZ| (slopes are
// below 1.13, |act(z)| <= |z|), then dZ in one more pass over the row.
template <bool GATED>
__global__ void __launch_bounds__(kDactThreads) dact_rows_kernel(const __grid_constant__ DactArgs g) {
  __shared__ float red[kDactThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const size_t m = blockIdx.x;
  const int nv = g.N >> 3;
  float top = 0.f;
  for (int v = threadIdx.x; v < nv; v += kDactThreads) {
    if (GATED) {
      float z[8];
      h8_to_f(__ldg(reinterpret_cast<const uint4*>(g.Z + m * g.N) + v), z);
      const uint2 h = __ldg(reinterpret_cast<const uint2*>(g.dY + m * (g.N >> 1)) + v);
      const float2 a = __half22float2(u32_as_h2(h.x)), b = __half22float2(u32_as_h2(h.y));
      const float dy[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = fmaxf(top, fabsf(dy[i]) * fmaxf(fabsf(z[2 * i]), fabsf(z[2 * i + 1])));
    } else {
      float d[8];
      h8_to_f(__ldg(reinterpret_cast<const uint4*>(g.dY + m * g.N) + v), d);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(d[i]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kDactThreads / 32; ++w) top = fmaxf(top, red[w]);
  // 2^e with top 2^e in [2^13, 2^14): |dZ m_n| 2^e stays below
  // 2^14 * 1.13 * 2.  A row of zeros, or one that holds an infinity, keeps e = 0.
  const uint32_t be = __float_as_uint(top) >> 23;
  const uint32_t se = (be == 0u || be == 255u) ? 127u : 267u - be;  // biased exponent of 2^e
  const uint32_t sc = se > 253u ? 253u : se;
  const float scale = __uint_as_float(sc << 23);
  if (threadIdx.x == 0) g.rowscale[m] = __uint_as_float((254u - sc) << 23);
  for (int v = threadIdx.x; v < nv; v += kDactThreads) {
    float d[8], c[8];
    dact_vec<GATED>(g, m, v, d);
    load_f8(g.cscale + 8 * v, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = (d[i] * scale) * chan_mant(__fmul_rn(c[i], g.cmul));
    reinterpret_cast<uint4*>(g.dZ + m * g.N)[v] = f_to_h8(d);
  }
}

// Partial column sums of dZ: thread t of CTA (x, y) owns the 8 channels of
// vector 128 x + t and the rows y, y + G, ...
template <bool GATED>
__global__ void __launch_bounds__(128) dact_columns_kernel(const __grid_constant__ DactArgs g) {
  griddep_launch_dependents();
  griddep_wait();
  const int v = blockIdx.x * 128 + threadIdx.x;
  if (v >= (g.N >> 3)) return;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int m = blockIdx.y; m < g.M; m += g.G) {
    float d[8];
    dact_vec<GATED>(g, m, v, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += d[i];
  }
  float4* p = reinterpret_cast<float4*>(g.part + static_cast<size_t>(blockIdx.y) * g.N) + 2 * v;
  p[0] = make_float4(s[0], s[1], s[2], s[3]);
  p[1] = make_float4(s[4], s[5], s[6], s[7]);
}

}  // namespace qlin
