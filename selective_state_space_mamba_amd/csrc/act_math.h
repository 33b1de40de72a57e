// act_math.h -- activations of the normalisation's and the matrix product's
// epilogues, and their derivatives.
#pragma once

#include "device_math.h"

namespace mscan {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3 };

// relu u if u > 0 else 0 (NaN stays NaN); silu u·sigmoid(u); gelu u·Φ(u), Φ the normal distribution's cdf
template <int ACT>
__device__ __forceinline__ float act_f(float u) {
  if constexpr (ACT == ACT_RELU) return u <= 0.f ? 0.f : u;
  if constexpr (ACT == ACT_SILU) return u * rcp(1.0f + ex2(-u * kLog2e));
  if constexpr (ACT == ACT_GELU) return 0.5f * u * (1.0f + erff(u * 0.70710678118654752440f));
  return u;
}

// relu' = [u > 0]; silu' = q(1 + u(1 - q)), q = sigmoid(u); gelu' = Φ(u) + u·φ(u)
template <int ACT>
__device__ __forceinline__ float act_d(float u) {
  if constexpr (ACT == ACT_RELU) return u > 0.f ? 1.f : 0.f;
  if constexpr (ACT == ACT_SILU) {
    const float q = rcp(1.0f + ex2(-u * kLog2e));
    return q * __builtin_fmaf(u, 1.0f - q, 1.0f);
  }
  if constexpr (ACT == ACT_GELU) {
    const float cdf = 0.5f * (1.0f + erff(u * 0.70710678118654752440f));
    return __builtin_fmaf(u * 0.39894228040143267794f, ex2(-0.5f * kLog2e * u * u), cdf);
  }
  return 1.f;
}

// The same with the activation known at run time (one for the whole launch).
__device__ __forceinline__ float act_any(float u, int act) {
  switch (act) {
    case ACT_RELU: return act_f<ACT_RELU>(u);
    case ACT_SILU: return act_f<ACT_SILU>(u);
    case ACT_GELU: return act_f<ACT_GELU>(u);
    default: return u;
  }
}
__device__ __forceinline__ float act_d_any(float u, int act) {
  switch (act) {
    case ACT_RELU: return act_d<ACT_RELU>(u);
    case ACT_SILU: return act_d<ACT_SILU>(u);
    case ACT_GELU: return act_d<ACT_GELU>(u);
    default: return 1.f;
  }
}

}  // namespace mscan
