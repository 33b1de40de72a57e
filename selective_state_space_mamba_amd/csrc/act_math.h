// act_math.h -- activations of the normalisation's and the matrix product's
// epilogues, and their derivatives.
#pragma once

#include "device_math.h"

namespace mscan {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3 };

// The standard normal cdf at u and e^{-u²/2}.  The tail beyond x = |u| is
// e^{-x²/2}·R(x), and R, which falls from 1/2 like 1/x, a polynomial without
// constant term in t = 1/(1 + 0.34 x): nine terms fitted here to R's definition,
// (1/2)·erfcx(x/sqrt 2), for the least relative error over x = 0..14 (4e-8, in
// these rounded coefficients).  So the tail keeps its relative accuracy down to
// the exponent's rounding (3e-6 at u = -8), and u·Φ(u) over normal arguments is
// off by 4e-8 like 0.5·u·(1 + erf).  The exponential serves the derivative too.
// (16384 x 768 x 1536 with gelu 63.3 us; 61.6 with five terms, which were right
// to 7.5e-8 absolute only, 92 with the library's erf, three times the instructions.)
__device__ __forceinline__ float normal_cdf(float u, float& e) {
  e = ex2(-0.5f * kLog2e * u * u);
  const float t = rcp(__builtin_fmaf(__builtin_fabsf(u), 0.34f, 1.0f));
  float p = __builtin_fmaf(t, -0.026120465f, 0.13949944f);
  p = __builtin_fmaf(t, p, -0.27313262f);
  p = __builtin_fmaf(t, p, 0.20218252f);
  p = __builtin_fmaf(t, p, -0.044718347f);
  p = __builtin_fmaf(t, p, 0.11535912f);
  p = __builtin_fmaf(t, p, 0.11519767f);
  p = __builtin_fmaf(t, p, 0.1361122f);
  p = __builtin_fmaf(t, p, 0.1356205f);
  const float tail = t * p * e;  // the cdf at -|u|
  return u < 0.f ? tail : 1.0f - tail;
}

// relu u if u > 0 else 0 (NaN stays NaN); silu u·sigmoid(u); gelu u·Φ(u), Φ the normal cdf
template <int ACT>
__device__ __forceinline__ float act_f(float u) {
  if constexpr (ACT == ACT_RELU) return u <= 0.f ? 0.f : u;
  if constexpr (ACT == ACT_SILU) return u * rcp(1.0f + ex2(-u * kLog2e));
  if constexpr (ACT == ACT_GELU) {
    float e;
    return u * normal_cdf(u, e);
  }
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
    float e;
    const float cdf = normal_cdf(u, e);
    return __builtin_fmaf(u * 0.39894228040143267794f, e, cdf);
  }
  return 1.f;
}

template <int ACT, int V>
__device__ __forceinline__ void act_each(float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = act_f<ACT>(v[j]);
}
// The same with the activation known at run time (one for the whole launch):
// one branch for all V values, whose instructions then interleave (in the
// matrix product's epilogue 16384 x 768 x 1536 with silu took 65 us with a
// branch a value, 54 so).
template <int V>
__device__ __forceinline__ void act_all(float (&v)[V], int act) {
  switch (act) {
    case ACT_RELU: act_each<ACT_RELU>(v); break;
    case ACT_SILU: act_each<ACT_SILU>(v); break;
    case ACT_GELU: act_each<ACT_GELU>(v); break;
    default: break;
  }
}
template <int ACT, int V>
__device__ __forceinline__ void act_d_each(float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = act_d<ACT>(v[j]);
}
template <int V>
__device__ __forceinline__ void act_d_all(float (&v)[V], int act) {
  switch (act) {
    case ACT_RELU: act_d_each<ACT_RELU>(v); break;
    case ACT_SILU: act_d_each<ACT_SILU>(v); break;
    case ACT_GELU: act_d_each<ACT_GELU>(v); break;
    default: act_d_each<ACT_NONE>(v);
  }
}

}  // namespace mscan
