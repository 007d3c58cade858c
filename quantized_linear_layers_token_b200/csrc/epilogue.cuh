// epilogue.cuh -- what the fused linear layers compute on each pre-activation
// value: bias, activation, residual, the gated product, and the activation's
// derivative for the backward pass.
//
//   relu(z) = max(z, 0)                 relu'  = [z > 0]
//   gelu(z) = z Phi(z)                  gelu'  = Phi(z) + z phi(z)
//   with Phi(-x) = exp(-x^2 / 2) P(t), t = 1 / (1 + 0.3 x), for x >= 0 and P a
//   polynomial of degree 8 without a constant term, fitted to
//   exp(x^2 / 2) Phi(-x) for the least relative error on [0, 14]: 1.5e-7
//   (a quarter of what the library's distribution function costs: measured
//   126 against 59 us for a 1000 x 11008 layer's product and epilogue)
//   gelu_tanh(z) = z p, p = 1 / (1 + exp(-2 u)), u = sqrt(2/pi) (z + 0.044715 z^3)
//                                       slope  = p + z p (1 - p) 2 u'
//   silu(z) = z p, p = 1 / (1 + exp(-z))       = p (1 + z (1 - p))
// with 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)).  All in fp32; the exponential
// and the quotient are the hardware approximations (a few units of 2^-22,
// far below half a step of the fp16 results), which reach 0 and z at the
// ends of the range without an overflow: exp(-2 u) = inf gives p = 0.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

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

__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

constexpr float kGeluTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluTanhB = 0.044715f;

// exp(-z^2 / 2) and Phi(z).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = __fdividef(1.f, fmaf(0.3f, fabsf(z), 1.f));
  e = __expf(-0.5f * z * z);
  float p = 0.03567487688139828f;
  p = fmaf(p, t, -0.15720349929292227f);
  p = fmaf(p, t, 0.2063541956658973f);
  p = fmaf(p, t, -0.05368424549759451f);
  p = fmaf(p, t, 0.12856192418724136f);
  p = fmaf(p, t, 0.09991340876296782f);
  p = fmaf(p, t, 0.12075396824859583f);
  p = fmaf(p, t, 0.11962929810635002f);
  const float q = p * t * e;
  return z < 0.f ? q : 1.f - q;
}

// act(z) of N values, the choice made once.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&z)[N]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float e;
        z[i] *= normal_cdf(z[i], e);
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = z[i] * sigmoid_f(kGeluTanhA * fmaf(kGeluTanhB * z[i], z[i] * z[i], z[i]));
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = z[i] * sigmoid_f(z[i]);
      break;
    default: break;
  }
}

// act(z) and act'(z) of N values.
template <int N>
__device__ __forceinline__ void act_slopes(int act, const float (&z)[N], float (&value)[N], float (&slope)[N]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        value[i] = z[i] < 0.f ? 0.f : z[i];
        slope[i] = z[i] > 0.f ? 1.f : 0.f;
      }
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float e;
        const float p = normal_cdf(z[i], e);
        value[i] = z[i] * p;
        slope[i] = fmaf(z[i] * 0.3989422804014327f, e, p);
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float z2 = z[i] * z[i];
        const float p = sigmoid_f(kGeluTanhA * fmaf(kGeluTanhB * z[i], z2, z[i]));
        value[i] = z[i] * p;
        slope[i] = fmaf(z[i] * p * (1.f - p), kGeluTanhA * fmaf(3.f * kGeluTanhB, z2, 1.f), p);
      }
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float p = sigmoid_f(z[i]);
        value[i] = z[i] * p;
        slope[i] = p * fmaf(z[i], 1.f - p, 1.f);
      }
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        value[i] = z[i];
        slope[i] = 1.f;
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
