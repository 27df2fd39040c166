// Activations of the experts' products and their slopes, on fp32 values.
#pragma once

#include <hip/hip_runtime.h>

#include "moe.h"
#include "moe_common.h"

namespace moe {

// the logistic function: for values that are rounded to bf16 on the hardware's exp2 and reciprocal
// (about 1 ulp of fp32 each), for fp32 ones with the library's exponential and a correct division
template <bool F32>
__device__ __forceinline__ float sigmoid_act(float x) {
  if (F32) return 1.0f / (1.0f + expf(-x));
  return sigmoid_f32(x);
}

constexpr float kGeluC = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// Phi(x), the normal distribution function, and e = exp(-x^2 / 2).  fp32: Phi(x) = erfc(-x / sqrt 2) / 2 keeps
// its digits where 1 + erf cancels.  For values that are rounded to bf16, the scaled tail exp(x^2 / 2)
// Phi(-|x|) as a polynomial of degree 6 in t = 1 / (1 + 0.32 |x|) without a constant term, fitted to it for
// the least largest relative error over 0 <= |x| <= 40 (1.2e-5, below 2^-16; the library's erfc took
// 111 us where this takes 75 in the gradient of 4585 rows of 12112, and its exponential is the density's too).
template <bool F32>
__device__ __forceinline__ float normal_cdf(float x, float& e) {
  if (F32) {
    e = expf(-0.5f * x * x);
    return 0.5f * erfcf(x * -0.70710678118654752f);
  }
  e = __builtin_amdgcn_exp2f(-0.72134752044448170f * x * x);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.32f, fabsf(x), 1.0f));
  float q = fmaf(-0.06677503883838654f, t, 0.13958698511123657f);
  q = fmaf(q, t, 0.049613259732723236f);
  q = fmaf(q, t, 0.12305139005184174f);
  q = fmaf(q, t, 0.12682823836803436f);
  q = fmaf(q, t, 0.1276896893978119f);
  q *= t * e;
  return x > 0.0f ? 1.0f - q : q;
}

// act(x):
//   none x | relu max(x, 0) | relu2 max(x, 0)^2 | gelu x Phi(x) | silu x s(x)
//   gelu_tanh x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2 = x s(2 sqrt(2/pi) (x + 0.044715 x^3))
template <bool F32>
__device__ __forceinline__ void act8(int act, float (&v)[8]) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];   // (NaN stays)
      break;
    case MOE_ACT_RELU2:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i] * v[i];
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float e;
        v[i] *= normal_cdf<F32>(v[i], e);
      }
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= sigmoid_act<F32>(kGeluC * (v[i] + kGeluB * v[i] * v[i] * v[i]));
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= sigmoid_act<F32>(v[i]);
      break;
    default: break;
  }
}

// v: pre-activations in, act(v) out; s: act'(v)
template <bool F32>
__device__ __forceinline__ void act8_slope(int act, float (&v)[8], float (&s)[8]) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[i] = v[i] > 0.0f ? 1.0f : (v[i] <= 0.0f ? 0.0f : v[i]);   // (NaN stays)
        v[i] = v[i] < 0.0f ? 0.0f : v[i];
      }
      break;
    case MOE_ACT_RELU2:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float r = v[i] < 0.0f ? 0.0f : v[i];
        s[i] = 2.0f * r;
        v[i] = r * r;
      }
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = v[i];
        float e;
        const float phi = normal_cdf<F32>(x, e);
        s[i] = phi + x * 0.39894228040143268f * e;
        v[i] = x * phi;
      }
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // (bounded: far out sg (1 - sg) is 0, and 0 times an infinity would be NaN)
        const float x = v[i], x2 = fminf(x * x, 1e30f);
        const float sg = sigmoid_act<F32>(kGeluC * (x + kGeluB * x2 * x));
        s[i] = sg + x * sg * (1.0f - sg) * (kGeluC * (1.0f + 3.0f * kGeluB * x2));
        v[i] = x * sg;
      }
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = v[i], sg = sigmoid_act<F32>(x);
        s[i] = sg * (1.0f + x * (1.0f - sg));
        v[i] = x * sg;
      }
      break;
    default:
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 1.0f;
      break;
  }
}

}  // namespace moe
