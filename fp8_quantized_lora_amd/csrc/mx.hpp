// Microscaled formats: blocks of 32 elements along a row with a power of two each,
// held as an E8M0 byte (exponent + 127).
//
// FP4 (E2M1 codes, two a byte): the exponent is floor(log2(amax)) - 2 of the
// block's largest finite magnitude, as the OCP microscaling specification has it:
// the largest element lies in [4, 8) and saturates at 6.
// 8-bit checkpoints (E4M3 codes): the smallest exponent with amax <= 448 2^e: no
// element saturates, at the price of half a binade for those blocks whose largest
// element lies in (448, 512).
// A block without a finite non-zero element has exponent 0 (byte 127).  Infinities and NaN
// have no part in the exponent: an infinity becomes the largest code under its block's
// finite neighbours' exponent, however small those are, and E2M1 has no NaN.
#pragma once

#include "common.hpp"
#include "mx_layout.hpp"

namespace falq {

// 2^e, -127 <= e <= 127 (2^-127 is subnormal)
__device__ __forceinline__ float exp2_int(int e) {
  return e > -127 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << 22);
}

// two E4M3 codes of a word by 2^(byte - 127): one instruction, which reads the scale's
// exponent field alone (0: 2^-127; 255: NaN).  With a multiplication of its own instead
// the norm's backward, which decodes each element twice, takes longer: 8192 x 5120 with
// float32 dy 85 us, 78 so; 8192 x 4100 85 and 75.
__device__ __forceinline__ float2 dec2_e8m0(uint32_t word, bool hi, uint32_t byte) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const float s = __uint_as_float(byte << 23);
  const v2f v = hi ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word, s, true)
                   : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word, s, false);
  return make_float2(v.x, v.y);
}

// exponents for a block whose largest finite magnitude has these bits
__device__ __forceinline__ int mx_exp_fp4(uint32_t mag) {
  if (mag == 0) return 0;
  const int e = __builtin_amdgcn_frexp_expf(__uint_as_float(mag)) - 3;
  return e < -127 ? -127 : e;
}
__device__ __forceinline__ int mx_exp_e4m3(uint32_t mag) {
  if (mag == 0) return 0;
  const float m = __uint_as_float(mag);            // f 2^E, 0.5 <= f < 1; 448 = 0.875 2^9
  const bool low = __builtin_amdgcn_frexp_mantf(m) <= 0.875f;
  const int e = __builtin_amdgcn_frexp_expf(m) - (low ? 9 : 8);
  return e < -127 ? -127 : e;
}

// eight values by 2^-e -> eight FP4 codes (value 0 in the low bits): to nearest, ties to
// the even code; larger ones and infinities saturate at 6, a NaN gives a zero
__device__ __forceinline__ uint32_t enc8_fp4(const float (&v)[8], int e) {
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = __builtin_isnan(v[i]) ? copysignf(0.0f, v[i]) : v[i];
  const float s = __uint_as_float((uint32_t)(e + 127) << 23);    // (its exponent field counts)
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[0], a[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[2], a[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[4], a[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[6], a[7], s, 3);
}
// eight codes by 2^(byte - 127)
__device__ __forceinline__ void dec8_fp4(uint32_t w, uint32_t byte, float (&v)[8]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const float s = __uint_as_float(byte << 23);
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
  const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
  const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
  const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}

// the largest finite magnitude of eight values, as ordered bits; over the four lanes
// of a block of 32
__device__ __forceinline__ uint32_t mag8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = max(m, a < 0x7F800000u ? a : 0u);
  }
  return m;
}
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  // lanes 1 0 3 2, then 2 3 0 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
}

}  // namespace falq
