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

// act(x):
//   none x | relu max(x, 0) | relu2 max(x, 0)^2 | gelu x Phi(x) | silu x s(x)
//   gelu_tanh x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2 = x s(2 sqrt(2/pi) (x + 0.044715 x^3))
// Phi(x) = erfc(-x / sqrt 2) / 2 keeps its digits where 1 + erf cancels.
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
      for (int i = 0; i < 8; ++i) v[i] = 0.5f * v[i] * erfcf(v[i] * -0.70710678118654752f);
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
        s[i] = v[i] > 0.0f ? 1.0f : 0.0f;
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
        const float phi = 0.5f * erfcf(x * -0.70710678118654752f);
        const float e = F32 ? expf(-0.5f * x * x) : __builtin_amdgcn_exp2f(-0.72134752044448170f * x * x);
        s[i] = phi + x * 0.39894228040143268f * e;
        v[i] = x * phi;
      }
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = v[i], x2 = x * x;
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
