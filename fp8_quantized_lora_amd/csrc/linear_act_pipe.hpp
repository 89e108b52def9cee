// The FP8 product with an epilogue in tiles of four waves: see linear_act.hip.
//
// A wave holds a quarter of the tile (128 x 128 of 256 x 256: 256 accumulation
// registers) and the fragments of one K step, so an LDS byte feeds up to eight
// products where the eight waves of linear_act_tile feed four.  Its quarter falls
// into quarters again, (A0, B0), (A0, B1), (A1, B1), (A1, B0): from one to the next
// one half of the fragments stays, and the half that is free takes the fragments
// that come after, so every LDS read is issued a quarter (512 cycles) before its
// use and the matrix cores do not wait for it.  The next step goes round the
// other way, from B1.
//
// The loads into LDS follow the same order: a slot of the LDS is what half a K step
// reads (half the rows of A and of B, a pair), a ring of three to five slots keeps
// the loads of the next two to four half steps under way, and one barrier for a
// half step says both that its pair has arrived and that the last one's slot is
// free.  4096 x 4096 x 4096: 51 us, 54 with eight waves and two stages; 8192 x 8192
// x 8192 372 and 430 (395 with a ring of two whole steps).
//
// Tiles of 256 x 320 and 256 x 256 have a CU to themselves; those up to 256 x 128
// take half of its LDS and registers, and one workgroup's epilogue runs under the
// other's products: 8192 x 10240 x 4096 with gelu and z 279 us in 256 x 128, 297 in
// 256 x 256 (331 with one workgroup of 256 x 128 on a CU).
#pragma once

#include "linear_act_tile.hpp"

namespace falq {
namespace {

// load16_to_lds with the address as a scalar base and a lane's 32-bit offset
__device__ __forceinline__ void load16_to_lds_at(const uint8_t* base, uint32_t off,
                                                 uint32_t lds_addr) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const uint64_t s = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(p >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)p);
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(s), "{m0}"(lds_addr)
               : "memory");
}

// d += a b^T of a 16 x 16 block, d in the same registers throughout (of the
// accumulation half of the file, ACC, or the other): left to itself the compiler
// moves the accumulators of a large tile through others at every loop turn
template <bool ACC>
__device__ __forceinline__ void mfma_in_place(v4f& d, const v8i& a, const v8i& b) {
  if constexpr (ACC)
    asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0" : "+a"(d) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x128_f8f6f4 %0, %1, %2, %0" : "+v"(d) : "v"(a), "v"(b));
}
// whether column block j of MB rows' blocks lies there: 64 blocks fill it
template <int MB>
constexpr bool in_acc(int j) {
  return (j + 1) * MB <= 64;
}

// f(0), ..., f(N - 1), each index a constant of its type
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}
#define FALQ_INLINE __attribute__((always_inline))

// d += a b^T of 16 x 16 blocks for every row fragment of a and column fragment of
// b; with(t) goes between product t and the next
template <int I0, int J0, int MB, int NB, int HM, int HN, class F>
__device__ __forceinline__ void quarter(v4f (&acc)[MB][NB], const v8i (&a)[HM],
                                        const v8i (&b)[HN], F&& with) {
  each<HM * HN>([&](auto t) FALQ_INLINE {
    constexpr int T = decltype(t)::value;
    mfma_in_place<in_acc<MB>(J0 + T % HN)>(acc[I0 + T / HN][J0 + T % HN], b[T % HN], a[T / HN]);
    with(t);
    __builtin_amdgcn_sched_barrier(0);
  });
}

// Between an asm product and whatever else may touch its result (a copy, where
// the compiler sees fit) pass the product's eight passes, which the compiler,
// not knowing the instruction, does not wait for: to be called where blocks of
// code meet, for copies arise there.
template <int MB, int NB>
__device__ __forceinline__ void settle(v4f (&acc)[MB][NB]) {
  asm volatile("s_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (in_acc<MB>(j))
        asm volatile("" : "+a"(acc[i][j]));
      else
        asm volatile("" : "+v"(acc[i][j]));
    }
}

template <class C, int PER_CU, class OT, bool STREAM>
__global__ __launch_bounds__(C::kThreads, PER_CU) void linear_act_pipe(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, Epilogue ep) {
  constexpr int BK = C::BK, MB = C::MB, NB = C::NB, HM = MB / 2, HN = NB / 2;
  // a slot: half the rows of either operand for one K step
  constexpr int UA = C::BM / 2 * BK, SLOT = UA + C::BN / 2 * BK;
  constexpr int FIT = 160 * 1024 / PER_CU / SLOT, SLOTS = FIT < 5 ? FIT : 5, AHEAD = SLOTS - 2;
  constexpr int LA = C::AI / 2, LB = C::BI / 2, LPP = LA + LB;
  static_assert(C::AI % 2 == 0 && C::BI % 2 == 0 && C::NW == 4, "whole loads per slot");
  static_assert(SLOTS >= 3, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[SLOTS * SLOT];
  int tm, tn;
  gemm::tile_of(gemm::xcd_remap((int)blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = __builtin_amdgcn_readfirstlane(tm * C::BM);
  const int n0 = __builtin_amdgcn_readfirstlane(tn * C::BN);
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = w / C::WGN, wn = w % C::WGN;
  const int nk = K / BK, rem = K % BK, all = nk + (rem > 0), last = 2 * all - 1;

  v4f acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // direct loads: the tile's first row as a scalar address, a lane's row (clamped
  // into the matrix) and swizzled chunk as its offset.  Half h of an operand is
  // half h of each wave's rows.
  const uint8_t* tA = A + (int64_t)m0 * K;
  const uint8_t* tB = B + (int64_t)n0 * K;
  const int lrow = lane >> 3, lslot = lane & 7;
  uint32_t vA[2][LA], vB[2][LB];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int j = 0; j < LA; ++j) {
      const int r = (w * LA + j) * 8 + lrow, row = (r / (C::WTM / 2) * 2 + h) * (C::WTM / 2) +
                                                   r % (C::WTM / 2);
      vA[h][j] = (uint32_t)min(row, M - 1 - m0) * (uint32_t)K + (lslot ^ gemm::dma::swz(r)) * 16;
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      const int r = (w * LB + j) * 8 + lrow, row = (r / (C::WTN / 2) * 2 + h) * (C::WTN / 2) +
                                                   r % (C::WTN / 2);
      vB[h][j] = (uint32_t)min(row, N - 1 - n0) * (uint32_t)K + (lslot ^ gemm::dma::swz(r)) * 16;
    }
  }
  const uint32_t ldsA = lds_offset(smem) + w * LA * 1024;
  const uint32_t ldsB = lds_offset(smem) + UA + w * LB * 1024;
  // load J of the wave's LPP: half HA of A's and half HB of B's rows, whole step kt
  auto load = [&](auto ha, auto hb, auto j, int kt, int slot) FALQ_INLINE {
    constexpr int J = decltype(j)::value;
    if constexpr (J < LA)
      load16_to_lds_at(tA + (int64_t)kt * BK, vA[decltype(ha)::value][J],
                       ldsA + slot * SLOT + J * 1024);
    else if constexpr (J < LPP)
      load16_to_lds_at(tB + (int64_t)kt * BK, vB[decltype(hb)::value][J - LA],
                       ldsB + slot * SLOT + (J - LA) * 1024);
  };
  // all of them, for any step; chunks past K load the row's last chunk
  auto fetch = [&](auto ha, auto hb, int kt, int slot) FALQ_INLINE {
    if (kt >= all) return;
    if (kt < nk) {
      each<LPP>([&](auto j) FALQ_INLINE { load(ha, hb, j, kt, slot); });
      return;
    }
    each<LPP>([&](auto j) FALQ_INLINE {
      constexpr int J = decltype(j)::value;
      if constexpr (J < LA) {
        const int co = (lslot ^ gemm::dma::swz((w * LA + J) * 8 + lrow)) * 16;
        load16_to_lds_at(tA + (int64_t)nk * BK, vA[decltype(ha)::value][J] - co + min(co, rem - 16),
                         ldsA + slot * SLOT + J * 1024);
      } else {
        const int co = (lslot ^ gemm::dma::swz((w * LB + J - LA) * 8 + lrow)) * 16;
        load16_to_lds_at(tB + (int64_t)nk * BK,
                         vB[decltype(hb)::value][J - LA] - co + min(co, rem - 16),
                         ldsB + slot * SLOT + (J - LA) * 1024);
      }
    });
  };
  // chunks past K of a slot of the step of rem bytes, once it has landed
  auto clear = [&](int slot) {
    for (int i = threadIdx.x; i < SLOT / 16; i += C::kThreads) {
      const int row = i >> 3, c = i & 7;                     // UA is a multiple of 16 rows
      if (c >= rem / 16)
        *reinterpret_cast<uint4*>(smem + slot * SLOT + row * BK +
                                  ((c ^ gemm::dma::swz(row & 15)) * 16)) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
  };

  const int r16 = lane & 15, g = lane >> 4, sw = gemm::dma::swz(r16);
  const int o0 = ((2 * g) ^ sw) * 16, o1 = ((2 * g + 1) ^ sw) * 16;
  const int offA = (wm * (C::WTM / 2) + r16) * BK, offB = UA + (wn * (C::WTN / 2) + r16) * BK;
  auto frag = [&](int at) FALQ_INLINE {
    return gemm::join(*reinterpret_cast<const uint4*>(smem + at + o0),
                      *reinterpret_cast<const uint4*>(smem + at + o1));
  };
  // with every second product a fragment of the group f at `at`
  auto read = [&](auto t, auto& f, int at) FALQ_INLINE {
    constexpr int T = decltype(t)::value, I = T / 2;
    if constexpr (T % 2 == 0 && I < sizeof(f) / sizeof(f[0])) f[I] = frag(at + I * 16 * BK);
  };
  v8i a0[HM], a1[HM], b0[HN], b1[HN];
  auto next = [](int slot) { return slot == SLOTS - 1 ? 0 : slot + 1; };
  // pair n, whose AHEAD successors are under way, is in its slot, and all waves are
  // done with pair n - 1
  auto arrive = [&](auto whole, int n, int slot, int kt) FALQ_INLINE {
    if constexpr (decltype(whole)::value) {
      __builtin_amdgcn_s_waitcnt(0x70 | ((AHEAD * LPP) & 0xF) | ((AHEAD * LPP) >> 4) << 14);
      barrier_no_drain();
    } else {
      settle(acc);
      __builtin_amdgcn_s_waitcnt(0xC07F);                    // lgkmcnt(0)
      wait_stages<AHEAD, LPP>(last - n);
      barrier_no_drain();
      if (kt == nk && rem) clear(slot);
    }
  };
  // K step k of parity P: slot is that of pair 2 k + 1
  auto step = [&](auto par, auto whole, int k, int& slot) FALQ_INLINE {
    constexpr bool P = decltype(par)::value, WHOLE = decltype(whole)::value;
    constexpr int jf = P ? HN : 0, jo = HN - jf;
    v8i(&f)[HN] = P ? b1 : b0;
    v8i(&o)[HN] = P ? b0 : b1;
    // the pairs that take the slots freed: SLOTS - 1 on from those read
    constexpr int D1 = SLOTS / 2, D2 = (SLOTS + 1) / 2, U = 2 * HM * HN / LPP;
    using HA1 = std::integral_constant<int, SLOTS % 2>;
    using HA2 = std::integral_constant<int, (SLOTS + 1) % 2>;
    using HB1 = std::integral_constant<int, (P + D1 + SLOTS) % 2>;
    using HB2 = std::integral_constant<int, (P + D2 + SLOTS + 1) % 2>;
    // load t / U of the pair's with every U-th product of a half step
    auto send = [&](auto t, auto first, auto ha, auto hb, int kt, int to) FALQ_INLINE {
      constexpr int T = decltype(t)::value + decltype(first)::value;
      if constexpr (WHOLE && T % U == 1)
        load(ha, hb, std::integral_constant<int, T / U>{}, kt, to);
    };
    using T0 = std::integral_constant<int, 0>;
    using T1 = std::integral_constant<int, HM * HN>;
    arrive(whole, 2 * k + 1, slot, k);
    int at = slot * SLOT, to = slot == 0 ? SLOTS - 1 : slot - 1;
    if constexpr (!WHOLE) fetch(HA1{}, HB1{}, k + D1, to);
    quarter<0, jf>(acc, a0, f, [&](auto t) FALQ_INLINE {
      read(t, o, at + offB);
      send(t, T0{}, HA1{}, HB1{}, k + D1, to);
    });
    quarter<0, jo>(acc, a0, o, [&](auto t) FALQ_INLINE {
      read(t, a1, at + offA);
      send(t, T1{}, HA1{}, HB1{}, k + D1, to);
    });
    to = slot;
    slot = next(slot);
    at = slot * SLOT;
    arrive(whole, 2 * k + 2, slot, k + 1);
    if constexpr (!WHOLE) fetch(HA2{}, HB2{}, k + D2, to);
    quarter<HM, jo>(acc, a1, o, [&](auto t) FALQ_INLINE {
      read(t, a0, at + offA);
      send(t, T0{}, HA2{}, HB2{}, k + D2, to);
    });
    quarter<HM, jf>(acc, a1, f, [&](auto t) FALQ_INLINE {
      read(t, o, at + offB);
      send(t, T1{}, HA2{}, HB2{}, k + D2, to);
    });
    slot = next(slot);
  };

  if (all > 0) {
    each<SLOTS>([&](auto q) FALQ_INLINE {
      constexpr int Q = decltype(q)::value;
      using HA = std::integral_constant<int, Q % 2>;
      using HB = std::integral_constant<int, (Q % 2 + Q / 2) % 2>;
      fetch(HA{}, HB{}, Q / 2, Q);
    });
    wait_stages<SLOTS - 1, LPP>(last);
    barrier_no_drain();
    if (nk == 0) clear(0);
#pragma unroll
    for (int i = 0; i < HM; ++i) a0[i] = frag(offA + i * 16 * BK);
#pragma unroll
    for (int j = 0; j < HN; ++j) b0[j] = frag(offB + j * 16 * BK);
  }
  const float scale = 1.0f / (ep.sa[0] * ep.sb[0]);
  __builtin_amdgcn_s_waitcnt(0xC07F);                        // lgkmcnt(0)
  int k = 0, slot = 1;
  for (; k + 1 + (SLOTS + 1) / 2 < nk; k += 2) {
    step(std::false_type{}, std::true_type{}, k, slot);
    step(std::true_type{}, std::true_type{}, k + 1, slot);
    settle(acc);
  }
  for (; k < all; k += 2) {
    step(std::false_type{}, std::false_type{}, k, slot);
    settle(acc);
    if (k + 1 < all) step(std::true_type{}, std::false_type{}, k + 1, slot);
    settle(acc);
  }
  settle(acc);
  __syncthreads();                                           // the slots are free
  tile_out<C, SLOTS * SLOT, OT, STREAM, false>(smem, acc, m0, n0, M, N, scale, ep, nullptr, 0);
}

}  // namespace
}  // namespace falq
