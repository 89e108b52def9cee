// The activations of a linear layer and their derivatives, in float32.
//
// gelu's normal distribution function comes from the rational-exponential
// form of Abramowitz and Stegun 7.1.26: for x >= 0
//     erfc(x) = (a1 t + a2 t^2 + ... + a5 t^5) exp(-x^2) + e,  t = 1 / (1 + p x),
// |e| <= 1.5e-7.  With x = |z| / sqrt(2) the exponential is exp(-z^2 / 2),
// which the derivative needs as well, so one exponential and one reciprocal
// serve both.  Phi(z) is therefore off by at most 7.5e-8 + roundings, about
// one float32 step of its largest value.
#pragma once

#include "common.hpp"

namespace falq {

enum Act : int { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4, kActs = 5 };

// 2^x and 1/x on the transcendental unit, about one float32 step each
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float logistic(float z) {
  return rcp_fast(1.0f + exp2_fast(-1.442695041f * z));
}

// logistic(x), and 1 - logistic(x) in `rest` without its cancellation (the
// bound keeps the exponential finite: inf * 0 does not arise)
__device__ __forceinline__ float logistic_pair(float x, float& rest) {
  const float e = exp2_fast(fminf(-1.442695041f * x, 126.0f));
  const float s = rcp_fast(1.0f + e);
  rest = e * s;
  return s;
}

// Phi(z), and exp(-z^2 / 2) in `ex`
__device__ __forceinline__ float normal_cdf(float z, float& ex) {
  const float a = fabsf(z);
  const float t = rcp_fast(fmaf(0.3275911f * 0.7071067812f, a, 1.0f));
  ex = exp2_fast(-0.7213475204f * z * z);
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  const float q = 0.5f * p * t * ex;           // Phi(-|z|)
  return z < 0.0f ? q : 1.0f - q;
}

constexpr float kTanhC = 0.7978845608f;        // sqrt(2 / pi)
constexpr float kTanhK = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kRelu) {
    return z < 0.0f ? 0.0f : z;
  } else if constexpr (ACT == kGelu) {
    float ex;
    return z * normal_cdf(z, ex);
  } else if constexpr (ACT == kGeluTanh) {     // (1 + tanh u) / 2 = logistic(2 u)
    return z * logistic(2.0f * kTanhC * z * fmaf(kTanhK * z, z, 1.0f));
  } else if constexpr (ACT == kSilu) {
    return z * logistic(z);
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kRelu) {
    return z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kGelu) {
    float ex;
    const float cdf = normal_cdf(z, ex);
    return fmaf(0.3989422804f * z, ex, cdf);
  } else if constexpr (ACT == kGeluTanh) {
    // the square is bounded so that 0 * inf does not arise for huge z
    const float z2 = fminf(z * z, 1e4f);
    float rest;
    const float s = logistic_pair(2.0f * kTanhC * z * fmaf(kTanhK, z2, 1.0f), rest);
    return fmaf(s * rest * (2.0f * kTanhC) * z, fmaf(3.0f * kTanhK, z2, 1.0f), s);
  } else if constexpr (ACT == kSilu) {
    float rest;
    const float s = logistic_pair(z, rest);
    return fmaf(s * z, rest, s);
  } else {
    return 1.0f;
  }
}

}  // namespace falq
