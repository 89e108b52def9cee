// Loads and stores of float32 / bfloat16 elements as floats, the activations
// and the fixed-order column sum that the row-wise operators share.
#pragma once

#include "common.hpp"

namespace falq {

typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

// E consecutive elements at p (16-byte aligned when E == 8)
template <int E>
__device__ __forceinline__ void load_elems(const float* p, float (&v)[E]) {
  if constexpr (E == 8) {
    const v4f a = *reinterpret_cast<const v4f*>(p), b = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
    static_assert(E == 1, "eight or one");
    v[0] = p[0];
  }
}
template <int E>
__device__ __forceinline__ void load_elems(const __bf16* p, float (&v)[E]) {
  if constexpr (E == 8) {
    const v8bf a = *reinterpret_cast<const v8bf*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)a[e];
  } else {
    static_assert(E == 1, "eight or one");
    v[0] = (float)p[0];
  }
}
template <int E>
__device__ __forceinline__ void store_elems(float* p, const float (&v)[E]) {
  if constexpr (E == 8) {
    *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f*>(p + 4) = v4f{v[4], v[5], v[6], v[7]};
  } else {
    p[0] = v[0];
  }
}
// bfloat16 results are rounded to nearest even, once
template <int E>
__device__ __forceinline__ void store_elems(__bf16* p, const float (&v)[E]) {
  if constexpr (E == 8) {
    v8bf a;
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = (__bf16)v[e];
    *reinterpret_cast<v8bf*>(p) = a;
  } else {
    p[0] = (__bf16)v[0];
  }
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

}  // namespace falq
