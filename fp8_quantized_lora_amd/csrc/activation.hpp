// The activations of a linear layer and their derivatives, in float32.
//
// gelu's normal distribution function: q(a) = Phi(-a) = exp(-a^2 / 2) P, a = |z|,
// P a minimax fit in relative error of exp(a^2 / 2) Phi(-a) up to a = 14.5, where the
// exponential underflows; Phi(z) is q for z < 0 and 1 - q above.
//
// For float32 P is a polynomial in v = -0.4 a / (1 + 0.4 a), P(0) = 1/2 (as float32
// numbers off by 3.9e-8, 2.5e-7 of the value; 0.4 keeps them small, so that
// Horner's roundings are).  v is formed as a product, since 1 / (1 + 0.4 a) - 1
// would carry the reciprocal's whole error to a = 0, where gelu is steep.  q is off
// by at most 1.3e-7 exp(-z^2 / 2) and the relative rounding of the exponential.
//
// Where the result is rounded to bfloat16, P = t R(t), t = 1 / (1 + c a): six terms
// for the value, off by 4.7e-6 of it (6.2e-6 with the roundings), a 600th of half a
// bfloat16 step; seven for the slope, whose sums stay float32, 1e-6 (1.6e-6).
// Products of 8192 x 11008 x 4096 and 1024 x 5120 x 5120 with gelu and z: 317 and
// 32.1 us with six terms, 324 and 32.8 with the nine of float32 (seven: 2 % and 1 %
// over six); bfloat16 backward of 8192 x 11008 and 4096 x 4096: 120.1 and 20.8 us
// with seven, 124.0 and 22.2 with nine.
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
// bound keeps the exponential finite: inf * 0 does not arise; a NaN passes it)
__device__ __forceinline__ float logistic_pair(float x, float& rest) {
  const float y = -1.442695041f * x;
  const float e = exp2_fast(y > 126.0f ? 126.0f : y);
  const float s = rcp_fast(1.0f + e);
  rest = e * s;
  return s;
}

// where every activation has reached its limit
constexpr float kFar = 100.0f;

// q of a = |z| with that many terms, and exp(-z^2 / 2)
struct NormalTail {
  float a, q, ex;
};
template <int TERMS>
__device__ __forceinline__ NormalTail normal_tail(float z) {
  static_assert(TERMS == 6 || TERMS == 7 || TERMS == 9, "fits");
  NormalTail n;
  // bounded where a is a factor (six terms: none), so that inf * 0 does not arise
  n.a = TERMS == 6 ? fabsf(z) : fminf(fabsf(z), kFar);
  n.ex = exp2_fast(-0.7213475204f * z * z);
  if constexpr (TERMS == 9) {
    const float v = -0.4f * n.a * rcp_fast(fmaf(0.4f, n.a, 1.0f));
    float p = fmaf(-0.0392525159f, v, -0.114942111f);
    p = fmaf(p, v, -0.0764153004f);
    p = fmaf(p, v, 0.00533220591f);
    p = fmaf(p, v, -0.113132618f);
    p = fmaf(p, v, -0.0515075214f);
    p = fmaf(p, v, 0.565024793f);
    p = fmaf(p, v, 0.997353077f);
    n.q = fmaf(p, v, 0.5f) * n.ex;
  } else if constexpr (TERMS == 7) {
    const float t = rcp_fast(fmaf(0.36f, n.a, 1.0f));
    float p = fmaf(0.0467824601f, t, -0.178826511f);
    p = fmaf(p, t, 0.179677546f);
    p = fmaf(p, t, 0.0274266712f);
    p = fmaf(p, t, 0.13940005f);
    p = fmaf(p, t, 0.141830385f);
    p = fmaf(p, t, 0.143708974f);
    n.q = p * t * n.ex;
  } else {
    const float t = rcp_fast(fmaf(0.31f, n.a, 1.0f));
    float p = fmaf(-0.0739291683f, t, 0.18045041f);
    p = fmaf(p, t, 0.0157446302f);
    p = fmaf(p, t, 0.133429825f);
    p = fmaf(p, t, 0.120441265f);
    p = fmaf(p, t, 0.123860702f);
    n.q = p * t * n.ex;
  }
  return n;
}

constexpr float kTanhC = 0.7978845608f;        // sqrt(2 / pi)
constexpr float kTanhK = 0.044715f;

// OT: the type that the value is rounded to
template <int ACT, class OT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kRelu) {
    return z < 0.0f ? 0.0f : z;
  } else if constexpr (ACT == kGelu) {
    const float q = normal_tail<std::is_same_v<OT, float> ? 9 : 6>(z).q;
    return z * (z < 0.0f ? q : 1.0f - q);
  } else if constexpr (ACT == kGeluTanh) {     // (1 + tanh u) / 2 = logistic(2 u)
    return z * logistic(2.0f * kTanhC * z * fmaf(kTanhK * z, z, 1.0f));
  } else if constexpr (ACT == kSilu) {
    return z * logistic(z);
  } else {
    return z;
  }
}

// z as the factor of a term that vanishes far out: what its other factor keeps of
// the bounds above (2^-126 for logistic_pair), or an infinity, would not vanish
// with z itself.  A NaN is carried by that other factor.
__device__ __forceinline__ float factor(float z) { return fminf(fmaxf(z, -kFar), kFar); }

template <int ACT, class OT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kRelu) {
    return z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kGelu) {
    // Phi(z) + z phi(z), which is q - a phi(a) at -a and 1 less that at a
    const NormalTail n = normal_tail<std::is_same_v<OT, float> ? 9 : 7>(z);
    const float low = fmaf(-0.3989422804f * n.a, n.ex, n.q);
    return z < 0.0f ? low : 1.0f - low;
  } else if constexpr (ACT == kGeluTanh) {
    // the square is bounded so that 0 * inf does not arise for huge z
    const float z2 = fminf(z * z, 1e4f);
    float rest;
    const float s = logistic_pair(2.0f * kTanhC * z * fmaf(kTanhK, z2, 1.0f), rest);
    return fmaf(s * rest * (2.0f * kTanhC) * factor(z), fmaf(3.0f * kTanhK, z2, 1.0f), s);
  } else if constexpr (ACT == kSilu) {
    float rest;
    const float s = logistic_pair(z, rest);
    return fmaf(s * factor(z), rest, s);
  } else {
    return 1.0f;
  }
}

}  // namespace falq
