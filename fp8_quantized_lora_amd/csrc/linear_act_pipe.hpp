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

// The products keep their accumulators in the same registers throughout
// (mma_in_place): left to itself the compiler moves those of a large tile through
// others at every loop turn.
// whether the accumulators of column block j of MB rows' blocks lie in the
// accumulation half, which 256 of a lane's registers fill
template <class ACC, int MB>
constexpr bool in_acc(int j) {
  return (j + 1) * MB * (int)sizeof(ACC) <= 64 * 16;
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

// d += a b^T of the blocks for every row fragment of a and column fragment of b
// (first of all blocks' first products, where a step takes several); with(t) goes
// between product t and the next.
template <class OP, int I0, int J0, int MB, int NB, int HM, int HN, class F>
__device__ __forceinline__ void quarter(typename OP::Acc (&acc)[MB][NB],
                                        const typename OP::Frag (&a)[HM],
                                        const typename OP::FragB (&b)[HN], F&& with) {
  typedef typename OP::Acc Acc;
  constexpr int BLOCKS = HM * HN;
  if constexpr (!OP::kConverted) {
    each<BLOCKS * OP::kProducts>([&](auto t) FALQ_INLINE {
      constexpr int T = decltype(t)::value, P = T % BLOCKS;
      OP::template mma_in_place<in_acc<Acc, MB>(J0 + P % HN), T / BLOCKS>(
          acc[I0 + P / HN][J0 + P % HN], b[P % HN], a[P / HN]);
      with(t);
      __builtin_amdgcn_sched_barrier(0);
    });
  } else {
    // the next product's operands are converted between this one's blocks
    constexpr int CA = OP::kConvertsA ? HM : 0;              // A's operands, then B's
    v4i ca[2][HM], cb[2][HN];
    auto convert = [&](auto to, auto o) FALQ_INLINE {
      constexpr int P = decltype(to)::value, O = decltype(o)::value;
      if constexpr (O < CA)
        ca[P % 2][O] = OP::template a_of<P>(a[O]);
      else
        cb[P % 2][O - CA] = OP::template b_of<P>(b[O - CA]);
    };
    using First = std::integral_constant<int, 0>;
    each<CA + HN>([&](auto o) FALQ_INLINE { convert(First{}, o); });
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 1");                                 // an operand's two wait states
    each<BLOCKS * OP::kProducts>([&](auto t) FALQ_INLINE {
      constexpr int T = decltype(t)::value, B = T % BLOCKS, P = T / BLOCKS;
      static_assert(in_acc<Acc, MB>(J0 + B % HN), "accumulators");
      const v4i& row = OP::kConvertsA ? ca[P % 2][B / HN] : OP::template a_of<P>(a[B / HN]);
      mfma_f16_in_place(acc[I0 + B / HN][J0 + B % HN], cb[P % 2][B % HN], row);
      if constexpr (P + 1 < OP::kProducts) {
        using Next = std::integral_constant<int, P + 1>;
        constexpr int O0 = B * (CA + HN) / BLOCKS, O1 = (B + 1) * (CA + HN) / BLOCKS;
        each<O1 - O0>([&](auto o) FALQ_INLINE {
          convert(Next{}, std::integral_constant<int, O0 + decltype(o)::value>{});
        });
      }
      with(t);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (B + 1 == BLOCKS) asm volatile("s_nop 1");
    });
  }
}

// Between an asm product and whatever else may touch its result (a copy, where
// the compiler sees fit) pass the product's eight passes, which the compiler,
// not knowing the instruction, does not wait for: to be called where blocks of
// code meet, for copies arise there.
template <int MB, int NB, class ACC>
__device__ __forceinline__ void settle(ACC (&acc)[MB][NB]) {
  asm volatile("s_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (in_acc<ACC, MB>(j))
        asm volatile("" : "+a"(acc[i][j]));
      else
        asm volatile("" : "+v"(acc[i][j]));
    }
}

// The LDS of pipe_product: a ring of slots, each half the rows of either operand
// for one K step (of a turned B the step's 64 rows of half the columns), and their
// exponent bytes, where there are any (8 a row).
template <class OP, class C, int PER_CU>
struct Ring {
  static constexpr int UA = C::BM / 2 * C::BK;
  static constexpr int CODES = UA + C::BN / 2 * (OP::kTurned ? 64 : C::BK);
  static constexpr int EXPS = 1024;                          // of half the rows, 8 each
  static constexpr int SLOT = CODES + (OP::kScaled ? 2 * EXPS : 0);
  static constexpr int FIT = 160 * 1024 / PER_CU / SLOT, SLOTS = FIT < 5 ? FIT : 5;
  static constexpr int kLds = SLOTS * SLOT;
  static_assert(SLOTS >= 3, "LDS");
};

// The tile at (m0, n0), wave-uniform, over K steps k_lo .. k_end - 1 (of all that K has;
// a k_lo that is not 0 with a turned B only): before() is called ahead of the loop,
// out(acc, what it gave, LDS) behind it, with the LDS (the ring's kLds) free.
//
// LEAN: one set of fragments of A instead of two, read between the quarters, where the
// registers do not hold two: the other workgroup of the CU multiplies meanwhile.
template <class OP, class C, int PER_CU, bool LEAN = false, class BEFORE, class OUT>
__device__ __forceinline__ void pipe_product(const uint8_t* __restrict__ A,
                                             const uint8_t* __restrict__ B, int M, int N, int K,
                                             int m0, int n0, int k_lo, int k_end,
                                             const Exponents& ex, BEFORE&& before, OUT&& out) {
  using R = Ring<OP, C, PER_CU>;
  typedef typename OP::Frag Frag;
  typedef typename OP::FragB FragB;
  // (declared here: through a pointer the compiler keeps an address per fragment, and
  // spills)
  __shared__ __attribute__((aligned(1024))) uint8_t smem[R::kLds];
  constexpr int BK = C::BK, BLK = OP::kBlock, MB = C::WTM / BLK, NB = C::WTN / BLK;
  constexpr int HM = MB / 2, HN = NB / 2, H = OP::kProducts;
  static_assert(MB % 2 == 0 && NB % 2 == 0, "quarters");
  constexpr int UA = R::UA, SLOT = R::SLOT, SLOTS = R::SLOTS, AHEAD = SLOTS - 2;
  constexpr bool TURNED = OP::kTurned;
  constexpr int LA = C::AI / 2, LB = TURNED ? C::BN / 2 * 64 / 1024 / 4 : C::BI / 2;
  constexpr int LPP = LA + LB;
  // turned: bytes and chunks of a row of half the columns, a wave's chunks of it, rows a load
  constexpr int RB = C::BN / 2, CPR = RB / 16, CPW = C::WTN / 2 / 16, RPL = 64 / CPR;
  static_assert(!TURNED || (LB * 4 * 1024 == RB * 64 && CPW == NB), "whole loads");
  static_assert(C::AI % 2 == 0 && C::BI % 2 == 0 && C::NW == 4, "whole loads per slot");
  static_assert(!OP::kScaled || (C::BM * 4 <= R::EXPS && C::BN * 4 <= R::EXPS), "exponents");
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = w / C::WGN, wn = w % C::WGN;
  // whole K steps, and the bytes or (turned) the rows of B of one that is not
  const int rows_b = TURNED ? ex.rows_b - k_lo * 64 : 0;
  const int nk = TURNED ? min(rows_b / 64, k_end - k_lo) : K / BK, rem = TURNED ? 0 : K % BK;
  const int all = min((K + BK - 1) / BK, k_end) - k_lo, last = 2 * all - 1;

  typename OP::Acc acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = typename OP::Acc{};

  // direct loads: the tile's first row as a scalar address, a lane's row (clamped
  // into the matrix) and swizzled chunk as its offset.  Half h of an operand is
  // half h of each wave's rows.
  const int64_t stepB = TURNED ? (int64_t)64 * N : BK;
  const uint8_t* tA = A + (int64_t)m0 * K + (int64_t)k_lo * BK;
  const uint8_t* tB = (TURNED ? B + n0 : B + (int64_t)n0 * K) + k_lo * stepB;
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
      if constexpr (TURNED) {
        const int r = (w * LB + j) * RPL + lane / CPR, c = (lane % CPR) ^ turned_swz<CPR>(r);
        vB[h][j] = (uint32_t)r * (uint32_t)N +
                   min(c / CPW * C::WTN + (h * CPW + c % CPW) * 16, N - 16 - n0);
        continue;
      }
      const int r = (w * LB + j) * 8 + lrow, row = (r / (C::WTN / 2) * 2 + h) * (C::WTN / 2) +
                                                   r % (C::WTN / 2);
      vB[h][j] = (uint32_t)min(row, N - 1 - n0) * (uint32_t)K + (lslot ^ gemm::dma::swz(r)) * 16;
    }
  }
  // exponents: wave 0 loads A's of a slot, wave 1 B's, two rows a lane
  const bool loads_e = OP::kScaled && w < 2;
  const uint8_t* tE = nullptr;
  uint32_t vE[2];
  int64_t estep = 0;
  if constexpr (OP::kScaled) {
    const int half = (w == 0 ? C::WTM : C::WTN) / 2, rows = w == 0 ? ex.rows_a : ex.rows_b;
    const int first = w == 0 ? m0 : n0, r = min(lane * 2, (w == 0 ? C::BM : C::BN) / 2 - 2);
    tE = (w == 0 ? ex.a : ex.b) + (int64_t)first * 8;
    estep = (int64_t)rows * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h)                             // rows is a multiple of 16
      vE[h] = (uint32_t)min((r / half * 2 + h) * half + r % half, rows - 2 - first) * 8;
  }
  const uint32_t ldsE = lds_offset(smem) + R::CODES + w * R::EXPS;
  const uint32_t ldsA = lds_offset(smem) + w * LA * 1024;
  const uint32_t ldsB = lds_offset(smem) + UA + w * LB * 1024;
  // load J of the wave's LPP: half HA of A's and half HB of B's rows, whole step kt
  auto load = [&](auto ha, auto hb, auto j, int kt, int slot) FALQ_INLINE {
    constexpr int J = decltype(j)::value;
    if constexpr (J < LA)
      load16_to_lds_at(tA + (int64_t)kt * BK, vA[decltype(ha)::value][J],
                       ldsA + slot * SLOT + J * 1024);
    else if constexpr (J < LPP)
      load16_to_lds_at(tB + kt * stepB, vB[decltype(hb)::value][J - LA],
                       ldsB + slot * SLOT + (J - LA) * 1024);
  };
  auto load_exponents = [&](auto ha, auto hb, int kt, int slot) FALQ_INLINE {
    if constexpr (OP::kScaled)
      if (loads_e)
        load16_to_lds_at(tE + kt * estep,
                         w == 0 ? vE[decltype(ha)::value] : vE[decltype(hb)::value],
                         ldsE + slot * SLOT);
  };
  // all of them, for any step; chunks past K load the row's last chunk
  auto fetch = [&](auto ha, auto hb, int kt, int slot) FALQ_INLINE {
    if (kt >= all) return;
    load_exponents(ha, hb, kt, slot);
    if (kt < nk) {
      each<LPP>([&](auto j) FALQ_INLINE { load(ha, hb, j, kt, slot); });
      return;
    }
    each<LPP>([&](auto j) FALQ_INLINE {
      constexpr int J = decltype(j)::value;
      if constexpr (TURNED && J < LA) {
        load(ha, hb, j, kt, slot);
      } else if constexpr (TURNED) {                         // rows past the last: the last
        const int r = (w * LB + J - LA) * RPL + lane / CPR;
        const int back = max(0, nk * 64 + r + 1 - rows_b);
        load16_to_lds_at(tB + kt * stepB,
                         vB[decltype(hb)::value][J - LA] - (uint32_t)back * (uint32_t)N,
                         ldsB + slot * SLOT + (J - LA) * 1024);
      } else if constexpr (J < LA) {
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
    for (int i = threadIdx.x; i < R::CODES / 16; i += C::kThreads) {
      const int row = i >> 3, c = i & 7;                     // UA is a multiple of 16 rows
      if (c >= rem / 16)
        *reinterpret_cast<uint4*>(smem + slot * SLOT + row * BK +
                                  ((c ^ gemm::dma::swz(row & 15)) * 16)) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
  };

  const int r = lane % BLK, g = lane / BLK;
  // the chunks of the lane's row, swizzled by the row's place among 16
  int o[OP::kParts];
#pragma unroll
  for (int p = 0; p < OP::kParts; ++p) o[p] = (OP::chunk(g, p) ^ gemm::dma::swz(r & 15)) * 16;
  const int offA = (wm * (C::WTM / 2) + r) * BK, offB = UA + (wn * (C::WTN / 2) + r) * BK;
  // the lane's exponents of fragment 0 of A and of B in a slot
  constexpr int EPL = 8 * BLK / 64;
  const int eA = R::CODES + (wm * (C::WTM / 2) + r) * 8 + EPL * g;
  const int eB = R::CODES + R::EXPS + (wn * (C::WTN / 2) + r) * 8 + EPL * g;
  // fragment I of a half of A, of B, of the slot that begins at byte `at`
  auto frag_at = [&](int codes, int exps) FALQ_INLINE {
    int e = 0;
    if constexpr (OP::kScaled)
      e = (int)*reinterpret_cast<const typename OP::Scales*>(smem + exps);
    uint4 q[OP::kParts];
#pragma unroll
    for (int p = 0; p < OP::kParts; ++p)
      q[p] = *reinterpret_cast<const uint4*>(smem + codes + o[p]);
    return OP::make(q, e);
  };
  auto fragA = [&](auto i, int at) FALQ_INLINE {
    constexpr int I = decltype(i)::value * BLK;
    return frag_at(at + offA + I * BK, at + eA + I * 8);
  };
  // turned: the lane's eight bytes of fragment 0 and 1 of a half of B
  int tB0 = 0, tB1 = 0;
  if constexpr (TURNED) {
    const int row = turned_row(lane), c = wn * CPW + ((lane >> 4) & 1), sz = turned_swz<CPR>(row);
    const int base = UA + (g * 8 + row) * RB + (lane & 1) * 8;
    tB0 = base + (c ^ sz) * 16;
    tB1 = base + ((c + 2) ^ sz) * 16;
  }
  auto fragB = [&](auto i, int at) FALQ_INLINE {
    constexpr int I = decltype(i)::value * BLK;
    if constexpr (TURNED) {
      static_assert(HN <= 2, "offsets");
      FragB f;
#pragma unroll
      for (int p = 0; p < OP::kParts; ++p)
        f.h[p] = read_turned(smem + at + (I == 0 ? tB0 : tB1) + p * 16 * RB);
      return f;
    } else
      return frag_at(at + offB + I * BK, at + eB + I * 8);
  };
  // with every second product a fragment of the group f (of 32 rows: every eighth)
  constexpr int EVERY = OP::kBlock == 16 ? 2 : HM * HN * H >= 16 ? 8 : 4;
  auto read = [&](auto t, auto& f, auto&& of, int at) FALQ_INLINE {
    constexpr int T = decltype(t)::value, I = T / EVERY, N = sizeof(f) / sizeof(f[0]);
    static_assert(T > 0 || (N - 1) * EVERY < HM * HN * H, "all within the quarter");
    if constexpr (T % EVERY == 0 && I < N) f[I] = of(std::integral_constant<int, I>{}, at);
  };
  Frag a0[HM], a_next[LEAN ? 1 : HM];
  FragB b0[HN], b1[HN];
  Frag(&a1)[HM] = *(Frag(*)[HM])(LEAN ? a0 : a_next);
  auto read_a = [&](int at) FALQ_INLINE {
    each<HM>([&](auto i) FALQ_INLINE { a0[decltype(i)::value] = fragA(i, at); });
  };
  auto next = [](int slot) { return slot == SLOTS - 1 ? 0 : slot + 1; };
  // until at most the loads of `ahead` pairs, at most A of them, are in flight
  auto wait_pairs = [&](auto most, int ahead) FALQ_INLINE {
    constexpr int A = decltype(most)::value;
    if (loads_e)
      wait_stages<A, LPP + 1>(ahead);
    else
      wait_stages<A, LPP>(ahead);
  };
  // pair n, whose AHEAD successors are under way, is in its slot, and all waves are
  // done with pair n - 1
  auto arrive = [&](auto whole, int n, int slot, int kt) FALQ_INLINE {
    if constexpr (decltype(whole)::value) {
      constexpr int MOST = AHEAD * LPP, MOST_E = AHEAD * (LPP + 1);
      if (loads_e)
        __builtin_amdgcn_s_waitcnt(0x70 | (MOST_E & 0xF) | (MOST_E >> 4) << 14);
      else
        __builtin_amdgcn_s_waitcnt(0x70 | (MOST & 0xF) | (MOST >> 4) << 14);
      barrier_no_drain();
    } else {
      settle(acc);
      __builtin_amdgcn_s_waitcnt(0xC07F);                    // lgkmcnt(0)
      wait_pairs(std::integral_constant<int, AHEAD>{}, last - n);
      barrier_no_drain();
      if (kt == nk && rem) clear(slot);
    }
  };
  // K step k of parity P: slot is that of pair 2 k + 1
  auto step = [&](auto par, auto whole, int k, int& slot) FALQ_INLINE {
    constexpr bool P = decltype(par)::value, WHOLE = decltype(whole)::value;
    constexpr int jf = P ? HN : 0, jo = HN - jf;
    FragB(&f)[HN] = P ? b1 : b0;
    FragB(&other)[HN] = P ? b0 : b1;
    // the pairs that take the slots freed: SLOTS - 1 on from those read
    constexpr int D1 = SLOTS / 2, D2 = (SLOTS + 1) / 2, U = 2 * HM * HN * H / LPP;
    static_assert(U > 0, "a product for each load");
    using HA1 = std::integral_constant<int, SLOTS % 2>;
    using HA2 = std::integral_constant<int, (SLOTS + 1) % 2>;
    using HB1 = std::integral_constant<int, (P + D1 + SLOTS) % 2>;
    using HB2 = std::integral_constant<int, (P + D2 + SLOTS + 1) % 2>;
    // load t / U of the pair's with every U-th product of a half step
    auto send = [&](auto t, auto first, auto ha, auto hb, int kt, int to) FALQ_INLINE {
      constexpr int T = decltype(t)::value + decltype(first)::value;
      if constexpr (WHOLE && T == 0) load_exponents(ha, hb, kt, to);
      if constexpr (WHOLE && T % U == (U > 1))
        load(ha, hb, std::integral_constant<int, T / U>{}, kt, to);
    };
    using T0 = std::integral_constant<int, 0>;
    using T1 = std::integral_constant<int, HM * HN * H>;
    arrive(whole, 2 * k + 1, slot, k);
    int at = slot * SLOT, to = slot == 0 ? SLOTS - 1 : slot - 1;
    if constexpr (!WHOLE) fetch(HA1{}, HB1{}, k + D1, to);
    quarter<OP, 0, jf>(acc, a0, f, [&](auto t) FALQ_INLINE {
      read(t, other, fragB, at);
      send(t, T0{}, HA1{}, HB1{}, k + D1, to);
    });
    quarter<OP, 0, jo>(acc, a0, other, [&](auto t) FALQ_INLINE {
      if constexpr (!LEAN) read(t, a1, fragA, at);
      send(t, T1{}, HA1{}, HB1{}, k + D1, to);
    });
    if constexpr (LEAN) read_a(at);
    to = slot;
    slot = next(slot);
    at = slot * SLOT;
    arrive(whole, 2 * k + 2, slot, k + 1);
    if constexpr (!WHOLE) fetch(HA2{}, HB2{}, k + D2, to);
    quarter<OP, HM, jo>(acc, a1, other, [&](auto t) FALQ_INLINE {
      if constexpr (!LEAN) read(t, a0, fragA, at);
      send(t, T0{}, HA2{}, HB2{}, k + D2, to);
    });
    quarter<OP, HM, jf>(acc, a1, f, [&](auto t) FALQ_INLINE {
      read(t, other, fragB, at);
      send(t, T1{}, HA2{}, HB2{}, k + D2, to);
    });
    if constexpr (LEAN) read_a(at);
    slot = next(slot);
  };

  if (all > 0) {
    each<SLOTS>([&](auto q) FALQ_INLINE {
      constexpr int Q = decltype(q)::value;
      using HA = std::integral_constant<int, Q % 2>;
      using HB = std::integral_constant<int, (Q % 2 + Q / 2) % 2>;
      fetch(HA{}, HB{}, Q / 2, Q);
    });
    wait_pairs(std::integral_constant<int, SLOTS - 1>{}, last);
    barrier_no_drain();
    if (nk == 0 && rem) clear(0);
    read_a(0);
    each<HN>([&](auto j) FALQ_INLINE { b0[decltype(j)::value] = fragB(j, 0); });
  }
  const auto kept = before();
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
  out(acc, kept, smem);
}

template <class OP, class C, int PER_CU, class OT, bool STREAM, bool LEAN = false>
__global__ __launch_bounds__(C::kThreads, PER_CU) void linear_act_pipe(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, Epilogue ep, Exponents ex) {
  int tm, tn;
  gemm::tile_of(gemm::xcd_remap((int)blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = __builtin_amdgcn_readfirstlane(tm * C::BM);
  const int n0 = __builtin_amdgcn_readfirstlane(tn * C::BN);
  pipe_product<OP, C, PER_CU, LEAN>(
      A, B, M, N, K, m0, n0, 0, INT32_MAX, ex, [&] { return scale_of<OP>(ep); },
      [&](const auto& acc, float scale, uint8_t* smem) {
        tile_out<C, Ring<OP, C, PER_CU>::kLds, OT, STREAM, false>(smem, acc, m0, n0, M, N, scale,
                                                                  ep, nullptr, 0);
      });
}

}  // namespace
}  // namespace falq
