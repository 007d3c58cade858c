// epilogue.cuh -- what the fused linear layers compute on each pre-activation
// value: bias, activation, residual, the gated product, and the activation's
// derivative for the backward pass.
//
//   relu(z) = max(z, 0)                 relu'  = [z > 0]
//   gelu(z) = z Phi(z)                  gelu'  = Phi(z) + z phi(z)
//   with Phi(-x) = exp(-x^2 / 2) P(t), t = 1 / (1 + 0.3 x), for x >= 0 and P a
//   polynomial of degree 8 without a constant term, fitted to
//   exp(x^2 / 2) Phi(-x) for the least relative error on [0, 14]: 1.5e-7, that
//   of the fit alone (a quarter of what the library's distribution function costs: measured
//   126 against 59 us for a 1000 x 11008 layer's product and epilogue)
//   gelu_tanh(z) = z p, p = 1 / (1 + exp(-2 u)), u = sqrt(2/pi) (z + 0.044715 z^3)
//                                       slope  = p + z p (1 - p) 2 u'
//   silu(z) = z p, p = 1 / (1 + exp(-z))       = p (1 + z (1 - p))
// with 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)).  All in fp32; the exponential
// and the reciprocal are the hardware approximations.  The exponential's
// argument x is rounded before it, so its relative error grows with x: about
// (2 + 1.2 |x|) 2^-23, x = z, 2 u or z^2 / 2 in GELU's tail.  Where a result is
// above fp16's smallest step (z > -5.5 for GELU, z > -20 for SiLU) |x| is below
// 20 and the error below 2^-18, against half a step of 2^-11.  The ends of the
// range are reached without an overflow: exp(-2 u) = inf gives p = 0.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "sm100.cuh"

namespace qlin {

enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// Epilogue variants of the GEMM kernels (template parameter).
enum : int {
  kEpiPlain = 0,  // Y = fp16(a (c' acc + comp))
  kEpiAct = 1,    // Z = a (c' acc + comp) + bias; Y = act(Z) + residual
  kEpiGated = 2   // the same Z; channels 2j, 2j + 1 are gate and up: Y[:, j] = act(Z[:, 2j]) Z[:, 2j + 1]
};

struct EpiArgs {
  const float* bias;         // [N] or null
  const uint16_t* residual;  // [M][N] or null (kEpiAct)
  uint16_t* Z;               // [M][N] or null: the pre-activation, kept for the backward pass
  int act;
};

// Eight fp16 values as four fp32 pairs, and back (rounded once).
__device__ __forceinline__ void h8_to_f2(const uint4 v, f32x2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
    f[e] = f2_pack(t.x, t.y);
  }
}
__device__ __forceinline__ uint4 f2_to_h8(const f32x2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 t = f2_unpack(f[e]);
    const __half2 h = __floats2half2_rn(t.x, t.y);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The arithmetic runs on fp32 pairs (one instruction for two values); the
// exponential and the reciprocal are a special-function operation a value.
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f32x2 ex2_pair(f32x2 x) {
  const float2 t = f2_unpack(x);
  return f2_pack(ex2_approx(t.x), ex2_approx(t.y));
}
__device__ __forceinline__ f32x2 rcp_pair(f32x2 x) {
  const float2 t = f2_unpack(x);
  return f2_pack(rcp_approx(t.x), rcp_approx(t.y));
}
// 1 / (1 + 2^x)
__device__ __forceinline__ f32x2 logistic2(f32x2 x) { return rcp_pair(f2_add(ex2_pair(x), f2_both(1.f))); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluTanhB = 0.044715f;

// z + 0.044715 z^3 from z and z^2
__device__ __forceinline__ f32x2 gelu_cubic(f32x2 z, f32x2 z2) {
  return f2_fma(f2_mul(z, f2_both(kGeluTanhB)), z2, z);
}

// exp(-z^2 / 2) and Phi(z).
__device__ __forceinline__ f32x2 normal_cdf(f32x2 z, f32x2& e) {
  const float2 v = f2_unpack(z);
  const f32x2 t = rcp_pair(f2_fma(f2_pack(fabsf(v.x), fabsf(v.y)), f2_both(0.3f), f2_both(1.f)));
  e = ex2_pair(f2_mul(f2_mul(z, z), f2_both(-0.5f * kLog2e)));
  f32x2 p = f2_both(0.03567487688139828f);
  p = f2_fma(p, t, f2_both(-0.15720349929292227f));
  p = f2_fma(p, t, f2_both(0.2063541956658973f));
  p = f2_fma(p, t, f2_both(-0.05368424549759451f));
  p = f2_fma(p, t, f2_both(0.12856192418724136f));
  p = f2_fma(p, t, f2_both(0.09991340876296782f));
  p = f2_fma(p, t, f2_both(0.12075396824859583f));
  p = f2_fma(p, t, f2_both(0.11962929810635002f));
  const float2 q = f2_unpack(f2_mul(f2_mul(p, t), e));
  return f2_pack(v.x < 0.f ? q.x : 1.f - q.x, v.y < 0.f ? q.y : 1.f - q.y);
}

// act(z) of N pairs, the choice made once.
template <int N>
__device__ __forceinline__ void act_pairs(int act, f32x2 (&z)[N]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 v = f2_unpack(z[i]);
        z[i] = f2_pack(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);
      }
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f32x2 e;
        z[i] = f2_mul(z[i], normal_cdf(z[i], e));
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i)
        z[i] = f2_mul(z[i], logistic2(f2_mul(gelu_cubic(z[i], f2_mul(z[i], z[i])), f2_both(-kGeluTanhA * kLog2e))));
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = f2_mul(z[i], logistic2(f2_mul(z[i], f2_both(-kLog2e))));
      break;
    default: break;
  }
}
// The same of N values, N even.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&z)[N]) {
  static_assert(N % 2 == 0, "values go in pairs");
  f32x2 v[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) v[i] = f2_pack(z[2 * i], z[2 * i + 1]);
  act_pairs<N / 2>(act, v);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 t = f2_unpack(v[i]);
    z[2 * i] = t.x;
    z[2 * i + 1] = t.y;
  }
}

// act(z) and act'(z) of N pairs, z kept in fp16.  A pre-activation past fp16's
// range arrives as an infinity and takes the limits -- slopes 0 and 1,
// act(-inf) = 0, act(inf) = inf -- so no product of an infinity and a vanishing
// factor may be formed: with LIMITS, z is held within +-65504 beside the
// factors that vanish (a NaN stays one through them).  Without, z is finite or
// NaN.
template <bool LIMITS, int N>
__device__ __forceinline__ void act_slopes(int act, const f32x2 (&z)[N], f32x2 (&value)[N], f32x2 (&slope)[N]) {
  const f32x2 one = f2_both(1.f);
  f32x2 above[N], inside[N];  // z from -65504 up; within +-65504
#pragma unroll
  for (int i = 0; i < N; ++i) {
    above[i] = inside[i] = z[i];
    if (LIMITS) {
      const float2 v = f2_unpack(z[i]);
      const float2 a = make_float2(fmaxf(v.x, -65504.f), fmaxf(v.y, -65504.f));
      above[i] = f2_pack(a.x, a.y);
      inside[i] = f2_pack(fminf(a.x, 65504.f), fminf(a.y, 65504.f));
    }
  }
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 v = f2_unpack(z[i]);
        value[i] = f2_pack(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);
        slope[i] = f2_pack(v.x > 0.f ? 1.f : 0.f, v.y > 0.f ? 1.f : 0.f);
      }
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f32x2 e;
        const f32x2 p = normal_cdf(z[i], e);
        value[i] = f2_mul(above[i], p);
        slope[i] = f2_fma(f2_mul(inside[i], f2_both(0.3989422804014327f)), e, p);
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const f32x2 z2 = f2_mul(inside[i], inside[i]);
        const f32x2 p = logistic2(f2_mul(gelu_cubic(z[i], z2), f2_both(-kGeluTanhA * kLog2e)));
        value[i] = f2_mul(above[i], p);
        const f32x2 q = f2_mul(f2_mul(inside[i], p), f2_fma(p, f2_both(-1.f), one));  // z p (1 - p)
        slope[i] = f2_fma(q, f2_fma(z2, f2_both(3.f * kGeluTanhA * kGeluTanhB), f2_both(kGeluTanhA)), p);
      }
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const f32x2 p = logistic2(f2_mul(z[i], f2_both(-kLog2e)));
        value[i] = f2_mul(above[i], p);
        slope[i] = f2_fma(f2_mul(inside[i], p), f2_fma(p, f2_both(-1.f), one), p);  // p + z p (1 - p)
      }
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        value[i] = z[i];
        slope[i] = one;
      }
  }
}

// Gated product of a channel pair held by two neighbouring lanes: the even
// lane holds the gate's, the odd lane the up projection's pre-activations of
// 2 n tokens.  After one exchange the even lane has both values of the first
// n tokens and the odd lane those of the last n; h[i] is act(gate) * up of
// token i (even lane) or n + i (odd lane).  `mask` names the lanes that call
// together (at least the pair).
template <int N2>
__device__ __forceinline__ void gated_pair(int act, const float (&z)[N2], bool odd, unsigned mask, float (&h)[N2 / 2]) {
  constexpr int n = N2 / 2;
  float up[n];
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const float send = odd ? z[i] : z[n + i];
    const float keep = odd ? z[n + i] : z[i];
    const float got = __shfl_xor_sync(mask, send, 1);
    h[i] = odd ? got : keep;
    up[i] = odd ? keep : got;
  }
  act_values<n>(act, h);
#pragma unroll
  for (int i = 0; i < n; ++i) h[i] *= up[i];
}

}  // namespace qlin
