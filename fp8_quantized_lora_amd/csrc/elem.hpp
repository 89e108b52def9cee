// Loads and stores of float32 / bfloat16 elements as floats, and wave sums, for
// the row-wise operators.
//
// E consecutive elements per lane: 4 or 8 (1 for rows shorter than that).  Stores
// of float32 take 4, 16 bytes a lane, so that a wave's store is one run of whole
// 128-byte lines: 32 bytes of a lane are two stores of half lines each, which the
// streaming hint below does not join again (backward of an activation, 8192 x
// 11008, fp32 gradients: 216 us with 8, 175 with 4).
#pragma once

#include "common.hpp"

#include <type_traits>

namespace falq {

typedef float v8f __attribute__((ext_vector_type(8)));

// Calls that touch more than the last-level cache holds (256 MB) read and write
// with the streaming hint (STREAM): what they leave in the caches would be
// displaced before anyone reads it, and the plain accesses cost it.  Smaller
// calls leave their results in the caches for the next one.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

// the vector of E elements of T in memory, aligned as T is: the 16-byte accesses
// work at any element, at full speed where the address is a multiple of 16
template <class T, int E>
struct VecOf {
  typedef T type;
};
template <>
struct VecOf<float, 4> {
  typedef v4f type __attribute__((aligned(4)));
};
template <>
struct VecOf<float, 8> {
  typedef v8f type __attribute__((aligned(4)));
};
template <>
struct VecOf<__bf16, 4> {
  typedef v2i type __attribute__((aligned(2)));
};
template <>
struct VecOf<__bf16, 8> {
  typedef v4i type __attribute__((aligned(2)));
};

// E elements as they lie in memory, for a load well ahead of its use
template <class T, int E>
struct Raw {
  typedef typename VecOf<T, E>::type V;
  V v;
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (STREAM && E > 1)
      v = __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
    else
      v = *reinterpret_cast<const V*>(p);
  }
  __device__ __forceinline__ void clear() { v = V{}; }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (E == 1) {
      return (float)v;
    } else if constexpr (std::is_same_v<T, float>) {
      return v[e];
    } else {                                   // bfloat16 is float32's upper half
      const uint32_t w = (uint32_t)v[e / 2];
      return __uint_as_float(e % 2 ? w & 0xFFFF0000u : w << 16);
    }
  }
};

// float32 parameters: eight in two vectors
template <int E>
__device__ __forceinline__ void load_elems(const float* p, float (&v)[E]) {
  if constexpr (E == 1) {
    v[0] = p[0];
  } else {
#pragma unroll
    for (int h = 0; h < E / 4; ++h) {
      const VecOf<float, 4>::type a = *reinterpret_cast<const VecOf<float, 4>::type*>(p + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * h + e] = a[e];
    }
  }
}
template <int E>
__device__ __forceinline__ void load_elems(const __bf16* p, float (&v)[E]) {
  Raw<__bf16, E> r;
  r.load(p);
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = r[e];
}

template <int E, bool STREAM = false>
__device__ __forceinline__ void store_elems(float* p, const float (&v)[E]) {
  if constexpr (E == 1) {
    p[0] = v[0];
  } else {
#pragma unroll
    for (int h = 0; h < E / 4; ++h) {
      const v4f a = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
      if constexpr (STREAM)
        __builtin_nontemporal_store(a, reinterpret_cast<VecOf<float, 4>::type*>(p + 4 * h));
      else
        *reinterpret_cast<VecOf<float, 4>::type*>(p + 4 * h) = a;
    }
  }
}
// bfloat16 results are rounded to nearest even, once
template <int E, bool STREAM = false>
__device__ __forceinline__ void store_elems(__bf16* p, const float (&v)[E]) {
  if constexpr (E == 1) {
    p[0] = (__bf16)v[0];
  } else {
    typedef __bf16 B __attribute__((ext_vector_type(E)));
    typedef typename VecOf<__bf16, E>::type V;
    B a;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = (__bf16)v[e];
    if constexpr (STREAM)
      __builtin_nontemporal_store(__builtin_bit_cast(V, a), reinterpret_cast<V*>(p));
    else
      *reinterpret_cast<V*>(p) = __builtin_bit_cast(V, a);
  }
}

// A lane's E elements of a row of d, from element i on.  ODD: d is no multiple of
// E, and the last piece ends with the row: it begins `over` elements early, and
// those are its neighbour's, to be left out of sums and stores.
template <int E, bool ODD>
struct Piece {
  uint32_t base;
  int over;
  bool any;
  __device__ __forceinline__ Piece(uint32_t i, uint32_t d) : base(i), over(0), any(i < d) {
    if (ODD && any && i + E > d) {
      over = (int)(i + E - d);
      base = d - E;
    }
  }
  __device__ __forceinline__ bool own(int e) const { return !ODD || e >= over; }
  template <bool STREAM = false, class T>
  __device__ __forceinline__ void store(T* row, const float (&v)[E]) const {
    if (!ODD || over == 0) {
      store_elems<E, STREAM>(row + base, v);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e >= over) row[base + e] = (T)v[e];
    }
  }
};

// Sum over the wave's 64 lanes, in every lane.  Within rows of 16 lanes by
// shifts, then across the rows: cross-lane operands of ordinary additions,
// where __shfl_xor would go through the LDS six times.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_moved(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF,
                                                        false));
}
// lanes 0 .. 15 only
__device__ __forceinline__ float row_sum_f32(float v) {
  v = add_moved<0x111, 0xF>(v);                // row_shr:1
  v = add_moved<0x112, 0xF>(v);                // row_shr:2
  v = add_moved<0x114, 0xF>(v);                // row_shr:4
  v = add_moved<0x118, 0xF>(v);                // row_shr:8
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 15));
}
__device__ __forceinline__ float wave_sum_f32(float v) {
  v = add_moved<0x111, 0xF>(v);                // row_shr:1
  v = add_moved<0x112, 0xF>(v);                // row_shr:2
  v = add_moved<0x114, 0xF>(v);                // row_shr:4
  v = add_moved<0x118, 0xF>(v);                // row_shr:8
  v = add_moved<0x142, 0xA>(v);                // lane 15 of rows 0, 2 to rows 1, 3
  v = add_moved<0x143, 0xC>(v);                // lane 31 to rows 2, 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

}  // namespace falq
