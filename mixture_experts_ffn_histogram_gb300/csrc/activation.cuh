// Activations of the linear layer and their derivatives, in fp32.
//
// EXACT false is for 16-bit results: the hardware exponential and reciprocal
// (2 ulp and 1), whose argument's rounding adds 1.2 ulp for each unit of it,
// and for gelu a polynomial for the normal distribution's tail (normal_cdf)
// with a relative error of at most 7e-6: 3% of half a step of fp16, 0.4% of one
// of bf16.  Below 2^-126 the exponential and the reciprocal are 0: silu and
// gelu_tanh at arguments of the sigmoid under -87.3, gelu under -13.2, where
// they lose less than 2e-36.  EXACT true is for fp32 results and uses the
// accurate functions.
#pragma once

#include "layer_common.cuh"

namespace moe {

template <bool EXACT>
__device__ __forceinline__ float act_sigmoid(float x) {
  if constexpr (EXACT) return 1.0f / (1.0f + expf(-x));
  else return rcp_fast(1.0f + exp2_fast(-kLog2e * x));
}

// Phi(z) and e^(-z^2/2).
template <bool EXACT>
__device__ __forceinline__ float2 normal_cdf(float z) {
  if constexpr (EXACT) {
    return make_float2(0.5f * erfcf(-0.70710678f * z), expf(-0.5f * z * z));
  } else {
    // Phi(-x) = e^(-x^2/2) t P(t) at t = 1 / (1 + 0.26 x): P minimises (linear
    // programme over 0 <= x <= 14) the largest error next to the smaller of
    // 2e-5 Phi(-x) and 1e-7; evaluated in fp32 it is off by at most 7e-6 of
    // Phi(-x), and 1.8e-7.
    const float t = rcp_fast(1.0f + 0.26f * fabsf(z));
    const float e = exp2_fast(z * z * (-0.5f * kLog2e));
    float poly = -0.07151548f;
    poly = 0.22278917f + t * poly;
    poly = -0.09589163f + t * poly;
    poly = 0.15729444f + t * poly;
    poly = 0.07749174f + t * poly;
    poly = 0.10623299f + t * poly;
    poly = 0.10359875f + t * poly;
    const float q = poly * t * e;
    return make_float2(z >= 0.0f ? 1.0f - q : q, e);
  }
}

constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

template <bool EXACT>
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z <= 0.0f ? 0.0f : z;  // NaN passes
    case MOE_ACT_GELU: return z * normal_cdf<EXACT>(z).x;
    case MOE_ACT_GELU_TANH:  // (1 + tanh u) / 2 = sigmoid(2 u)
      return z * act_sigmoid<EXACT>(kGeluA * z * (1.0f + kGeluB * z * z));
    case MOE_ACT_SILU: return z * act_sigmoid<EXACT>(z);
    default: return z;
  }
}

// The activation of N values at once: one branch on its kind.
template <bool EXACT, int N, int ACT>
__device__ __forceinline__ void act_run(float* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = act_value<EXACT>(v[i], ACT);
}
template <bool EXACT, int N>
__device__ __forceinline__ void act_all(float* v, int act) {
  switch (act) {
    case MOE_ACT_RELU: act_run<EXACT, N, MOE_ACT_RELU>(v); break;
    case MOE_ACT_GELU: act_run<EXACT, N, MOE_ACT_GELU>(v); break;
    case MOE_ACT_GELU_TANH: act_run<EXACT, N, MOE_ACT_GELU_TANH>(v); break;
    case MOE_ACT_SILU: act_run<EXACT, N, MOE_ACT_SILU>(v); break;
    default: break;
  }
}

template <bool EXACT>
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    case MOE_ACT_GELU: {
      const float2 c = normal_cdf<EXACT>(z);
      return c.x + 0.3989422804f * z * c.y;
    }
    case MOE_ACT_GELU_TANH: {
      const float s = act_sigmoid<EXACT>(kGeluA * z * (1.0f + kGeluB * z * z));
      const float d = s * (1.0f - s);  // 0 long before z * z overflows
      return d > 0.0f ? s + z * d * kGeluA * (1.0f + 3.0f * kGeluB * z * z) : s;
    }
    case MOE_ACT_SILU: {
      const float s = act_sigmoid<EXACT>(z);
      return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
  }
}

}  // namespace moe
