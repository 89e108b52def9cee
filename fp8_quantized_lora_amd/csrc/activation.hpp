// The activations of a linear layer and their derivatives, in float32.
//
// gelu's normal distribution function: Phi(-a) = exp(-a^2 / 2) P(v) for a = |z|,
// with v = -p a / (1 + p a) from 0 to -1 and P a polynomial, P(0) = 1/2.  Its
// coefficients are a minimax fit, in relative error, of exp(a^2 / 2) Phi(-a) up to
// a = 14.5, where the exponential underflows (as float32 numbers off by 3.9e-8,
// 2.5e-7 of the value); p = 0.4 keeps them small, so that Horner's roundings are.  v is formed as a
// product, since 1 / (1 + p a) - 1 would carry the reciprocal's whole error to
// a = 0, where gelu is steep.  exp(-z^2 / 2) is what the derivative needs as well,
// so one exponential and one reciprocal serve both.  Phi is off by at most
// 1.3e-7 exp(-z^2 / 2), the relative rounding of the exponential and 2^-24.
#pragma once

#include "common.hpp"

#include <type_traits>

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

// where every activation has reached its limit
constexpr float kFar = 100.0f;

// Phi(z), and exp(-z^2 / 2) in `ex`
__device__ __forceinline__ float normal_cdf(float z, float& ex) {
  constexpr float kP = 0.4f;
  const float a = fminf(fabsf(z), kFar);       // inf * 0 does not arise in v
  const float v = -kP * a * rcp_fast(fmaf(kP, a, 1.0f));
  ex = exp2_fast(-0.7213475204f * z * z);
  float p = fmaf(-0.0392525159f, v, -0.114942111f);
  p = fmaf(p, v, -0.0764153004f);
  p = fmaf(p, v, 0.00533220591f);
  p = fmaf(p, v, -0.113132618f);
  p = fmaf(p, v, -0.0515075214f);
  p = fmaf(p, v, 0.565024793f);
  p = fmaf(p, v, 0.997353077f);
  const float q = fmaf(p, v, 0.5f) * ex;       // Phi(-|z|)
  return z < 0.0f ? q : 1.0f - q;
}

// The same for results that are rounded to bfloat16: Phi(-a) = exp(-a^2 / 2) t
// R(t), t = 1 / (1 + p a), R a minimax fit in relative error, 4.7e-6 (6.2e-6 with
// the roundings): a 600th of half a bfloat16 step, at five operations fewer
// (8192 x 11008 x 4096 with gelu and z: 323 us, 328 with the form above).
__device__ __forceinline__ float normal_cdf_short(float z) {
  const float t = rcp_fast(fmaf(0.31f, fabsf(z), 1.0f));
  const float ex = exp2_fast(-0.7213475204f * z * z);
  float p = fmaf(-0.0739291683f, t, 0.18045041f);
  p = fmaf(p, t, 0.0157446302f);
  p = fmaf(p, t, 0.133429825f);
  p = fmaf(p, t, 0.120441265f);
  p = fmaf(p, t, 0.123860702f);
  const float q = p * t * ex;                  // Phi(-|z|)
  return z < 0.0f ? q : 1.0f - q;
}

constexpr float kTanhC = 0.7978845608f;        // sqrt(2 / pi)
constexpr float kTanhK = 0.044715f;

// OT: the type that the value is rounded to
template <int ACT, class OT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kRelu) {
    return z < 0.0f ? 0.0f : z;
  } else if constexpr (ACT == kGelu && !std::is_same_v<OT, float>) {
    return z * normal_cdf_short(z);
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
