// What the tiled products (linear_act_few.hpp, linear_act_tile.hpp,
// linear_act_pipe.hpp) multiply: E4M3 codes, E4M3 codes as float16, float16 by E4M3
// codes of the other orientation, or FP4 E2M1 codes with a power of two per block of 32.
// All count K in bytes, a step of 128 of them a row.  A fragment is a step of kBlock rows
// (16 or 32): a lane holds kParts chunks of 16 bytes of row lane % kBlock, chunk(g, p), g =
// lane / kBlock; which ones is free, as long as both operands' agree.
//
// Blocks of 32 x 32 take half the LDS reads of an instruction of 16 x 16 and, where
// an instruction of 16 x 16 has four passes (float16, FP4), are the only ones that one
// wave on a SIMD can issue without a pause: 2.4 PFLOP/s of float16 against 1.5, 9.1 of
// FP4 against 6.2 (2.2 and 8.7 with two waves).
//
// E4M3 in v_mfma_..._f8f6f4 is not exact: of eight products at a time, bits 2^-13
// below the largest are lost (4.5e-5 of a logit's spread where some channels are
// twenty times the others).  As float16, which holds every code, sums are float32's,
// at half the rate: the softmax's logits are formed so (E4M3AsF16), but for gradients in
// bfloat16.
#pragma once

#include "gemm_fp8_kernel.hpp"
#include "mx.hpp"

namespace falq {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4i as_v4i(uint4 v) {
  return v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
}

// make: a fragment of its chunks (and exponent bytes).
// mma: c + b a^T of a step.  mma_in_place<ACC, P>: product P of kProducts of it, with c
// in the same registers throughout (of the accumulation half of the file, ACC, or the
// other).
struct E4M3 {
  static constexpr int kBlock = 16, kParts = 2, kProducts = 1;
  static constexpr bool kScaled = false, kConverted = false, kTurned = false;
  typedef v4f Acc;
  typedef v8i Frag;
  typedef Frag FragB;
  static __device__ __forceinline__ int chunk(int g, int p) { return 2 * g + p; }
  static __device__ __forceinline__ Frag make(const uint4 (&q)[2], int) {
    return gemm::join(q[0], q[1]);
  }
  static __device__ __forceinline__ v4f mma(const Frag& b, const Frag& a, v4f c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, 0, 0, 0, 0);
  }
  template <bool ACC, int P>
  static __device__ __forceinline__ void mma_in_place(v4f& d, const Frag& b, const Frag& a) {
    if constexpr (ACC)
      asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0" : "+a"(d) : "v"(b), "v"(a));
    else
      asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0" : "+v"(d) : "v"(b), "v"(a));
  }
};

// N chunks
template <int N>
struct Chunks {
  v4i h[N];
};
template <int N>
__device__ __forceinline__ Chunks<N> chunks_of(const uint4 (&q)[N]) {
  Chunks<N> f;
#pragma unroll
  for (int i = 0; i < N; ++i) f.h[i] = as_v4i(q[i]);
  return f;
}

__device__ __forceinline__ v4f mfma_f16(v4i b, v4i a, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, b),
                                                __builtin_bit_cast(v8h, a), c, 0, 0, 0);
}
// (32 x 32: the accumulators are in the accumulation half wherever these are used)
__device__ __forceinline__ void mfma_f16_in_place(v16f& d, v4i b, v4i a) {
  asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+a"(d) : "v"(b), "v"(a));
}

// two and eight codes as float16
template <bool HI>
__device__ __forceinline__ int f16_pair_of_e4m3(int w) {
  return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)w, 1.0f, HI));
}
__device__ __forceinline__ v4i f16_of_e4m3(int lo, int hi) {
  return v4i{f16_pair_of_e4m3<false>(lo), f16_pair_of_e4m3<true>(lo), f16_pair_of_e4m3<false>(hi),
             f16_pair_of_e4m3<true>(hi)};
}
// half H of a chunk
template <int H>
__device__ __forceinline__ v4i f16_of_e4m3(v4i q) {
  return f16_of_e4m3(q[2 * H], q[2 * H + 1]);
}
struct E4M3AsF16 {
  static constexpr int kBlock = 16, kParts = 2;
  static constexpr bool kScaled = false, kTurned = false;
  typedef v4f Acc;
  typedef Chunks<2> Frag;
  typedef Frag FragB;
  static __device__ __forceinline__ int chunk(int g, int p) { return g + 4 * p; }
  static __device__ __forceinline__ Frag make(const uint4 (&q)[2], int) { return chunks_of(q); }
  static __device__ __forceinline__ v4f mma(const Frag& b, const Frag& a, v4f c) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      c = mfma_f16(f16_of_e4m3<0>(b.h[p]), f16_of_e4m3<0>(a.h[p]), c);
      c = mfma_f16(f16_of_e4m3<1>(b.h[p]), f16_of_e4m3<1>(a.h[p]), c);
    }
    return c;
  }
};
// kConverted: product P multiplies a_of<P>() and b_of<P>() of the fragments; kConvertsA:
// a_of is more than one of the fragment's registers.
struct E4M3AsF16Wide {
  static constexpr int kBlock = 32, kParts = 4, kProducts = 8;
  static constexpr bool kScaled = false, kConverted = true, kConvertsA = true, kTurned = false;
  typedef v16f Acc;
  typedef Chunks<4> Frag;
  typedef Frag FragB;
  static __device__ __forceinline__ int chunk(int g, int p) { return g + 2 * p; }
  static __device__ __forceinline__ Frag make(const uint4 (&q)[4], int) { return chunks_of(q); }
  template <int P>
  static __device__ __forceinline__ v4i a_of(const Frag& f) {
    return f16_of_e4m3<P % 2>(f.h[P / 2]);
  }
  template <int P>
  static __device__ __forceinline__ v4i b_of(const Frag& f) {
    return a_of<P>(f);
  }
};

// kTurned: A float16, 64 columns a step, times B itself, not its transpose: B's rows are
// the contraction's index, 64 of them a step (ex.rows_b in all), E4M3 codes that run
// along the outputs' columns.  They lie in LDS as in memory, and the transposing read
// gives each lane eight rows of its column: of the 16 lanes of a group, lane j names the
// eight bytes at row j / 2 and column 8 (j % 2) of a block of 8 rows x 16 columns, and
// lane n receives column n.
typedef __attribute__((address_space(3))) v2i lds_v2i;
__device__ __forceinline__ v2i read_turned(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)p);
}
// where a lane's row lies within eight, and chunk c of a row of CPR chunks of 16 bytes:
// eight rows' chunks of one column in different banks
__device__ __forceinline__ int turned_row(int lane) { return (lane & 15) >> 1; }
template <int CPR>
__device__ __forceinline__ int turned_swz(int row) {
  static_assert(CPR == 8 || CPR == 4, "rows of 128 or 64 bytes");
  return CPR == 8 ? row & 7 : (row >> 1) & 3;
}
// parts: a lane's eight rows, 8 g on, of each 32 (blocks of 16) or 16 (of 32) of a step
template <int N>
struct TurnedParts {
  v2i h[N];
};
struct F16ByE4M3 {
  static constexpr int kBlock = 16, kParts = 2;
  static constexpr bool kScaled = false, kTurned = true;
  typedef v4f Acc;
  typedef Chunks<2> Frag;
  typedef TurnedParts<2> FragB;
  static __device__ __forceinline__ int chunk(int g, int p) { return g + 4 * p; }
  static __device__ __forceinline__ Frag make(const uint4 (&q)[2], int) { return chunks_of(q); }
  static __device__ __forceinline__ v4f mma(const FragB& b, const Frag& a, v4f c) {
#pragma unroll
    for (int p = 0; p < 2; ++p) c = mfma_f16(f16_of_e4m3(b.h[p][0], b.h[p][1]), a.h[p], c);
    return c;
  }
};
struct F16ByE4M3Wide {
  static constexpr int kBlock = 32, kParts = 4, kProducts = 4;
  static constexpr bool kScaled = false, kConverted = true, kConvertsA = false, kTurned = true;
  typedef v16f Acc;
  typedef Chunks<4> Frag;
  typedef TurnedParts<4> FragB;
  static __device__ __forceinline__ int chunk(int g, int p) { return g + 2 * p; }
  static __device__ __forceinline__ Frag make(const uint4 (&q)[4], int) { return chunks_of(q); }
  template <int P>
  static __device__ __forceinline__ v4i a_of(const Frag& f) {
    return f.h[P];
  }
  template <int P>
  static __device__ __forceinline__ v4i b_of(const FragB& f) {
    return f16_of_e4m3(f.h[P][0], f.h[P][1]);
  }
};

// s: the exponent bytes of the lane's chunks, which mx_layout.hpp puts side by side
struct Fp4 {
  static constexpr int kBlock = 16, kParts = 2;
  static constexpr bool kScaled = true, kTurned = false;
  typedef uint16_t Scales;
  typedef v4f Acc;
  struct Frag {
    v4i h[2];
    int s;
  };
  typedef Frag FragB;
  static __device__ __forceinline__ int chunk(int g, int p) { return mx_block_at(2 * g + p); }
  static __device__ __forceinline__ Frag make(const uint4 (&q)[2], int s) {
    return {{as_v4i(q[0]), as_v4i(q[1])}, s};
  }
  static __device__ __forceinline__ v8i wide(v4i v) {
    return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
  }
  static __device__ __forceinline__ v4f mma(const Frag& b, const Frag& a, v4f c) {
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(b.h[0]), wide(a.h[0]), c, 4, 4, 0,
                                                         b.s, 0, a.s);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(b.h[1]), wide(a.h[1]), c, 4, 4, 1,
                                                            b.s, 1, a.s);
  }
};
struct Fp4Wide {
  static constexpr int kBlock = 32, kParts = 4, kProducts = 4;
  static constexpr bool kScaled = true, kConverted = false, kTurned = false;
  typedef uint32_t Scales;
  typedef v16f Acc;
  struct Frag {
    v4i h[4];
    int s;
  };
  typedef Frag FragB;
  static __device__ __forceinline__ int chunk(int g, int p) { return mx_block_at(4 * g + p); }
  static __device__ __forceinline__ Frag make(const uint4 (&q)[4], int s) {
    return {{as_v4i(q[0]), as_v4i(q[1]), as_v4i(q[2]), as_v4i(q[3])}, s};
  }
  // byte P of the scales, by both operands' selects
#define FALQ_FP4(SEL)                                                                          \
  asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL " cbsz:4 blgp:4" \
               : "+a"(d)                                                                       \
               : "v"(b.h[P]), "v"(a.h[P]), "v"(b.s), "v"(a.s))
  template <bool ACC, int P>
  static __device__ __forceinline__ void mma_in_place(v16f& d, const Frag& b, const Frag& a) {
    static_assert(ACC, "accumulators");
    if constexpr (P == 0)
      FALQ_FP4("op_sel_hi:[0,0,0]");
    else if constexpr (P == 1)
      FALQ_FP4("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
    else if constexpr (P == 2)
      FALQ_FP4("op_sel_hi:[1,1,0]");
    else
      FALQ_FP4("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
  }
#undef FALQ_FP4
};

// Where the exponent bytes of a product's operands lie (kScaled; mx_layout.hpp), with
// their rows rounded up to multiples of 16.  rows_b: also the rows of a turned B.
struct Exponents {
  const uint8_t* a;
  const uint8_t* b;
  int rows_a, rows_b;
};

}  // namespace falq
