// The FP8 product with an epilogue in tiles: see linear_act.hip.
#pragma once

#include "linear_act_few.hpp"

namespace falq {
namespace {

template <int BM_, int BN_, int WGM_, int WGN_, int S_ = 2>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, BK = 128, S = S_;
  static constexpr int NW = WGM * WGN, kThreads = NW * 64;
  static constexpr int WTM = BM / WGM, WTN = BN / WGN, MB = WTM / 16, NB = WTN / 16;
  static constexpr int STAGE = (BM + BN) * BK;
  static constexpr int AI = BM / 8 / NW, BI = BN / 8 / NW;   // 1 KB loads per wave and stage
  static constexpr int LPS = AI + BI;
  // the epilogue: rows of a wave's sub-tile per pass through its part of the LDS
  static constexpr int pass_of(int p, int lds) {
    return p * WTN * 4 * NW <= lds ? p : pass_of(p / 2, lds);
  }
  static_assert(AI * 8 * NW == BM && BI * 8 * NW == BN, "whole loads");
  static_assert(S * STAGE <= 160 * 1024, "LDS");
};

// waits until at most N vector-memory instructions of the wave are in flight
template <int N>
__device__ __forceinline__ void wait_vmem_at_most() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
// at most ahead * LPS, ahead <= A
template <int A, int LPS>
__device__ __forceinline__ void wait_stages(int ahead) {
  if constexpr (A == 0) {
    wait_vmem_at_most<0>();
  } else {
    if (ahead >= A)
      wait_vmem_at_most<A * LPS>();
    else
      wait_stages<A - 1, LPS>(ahead);
  }
}

// A wave's accumulators of rows first .. first + PASS - 1 into its part of the LDS,
// four columns of a row at slot(row, column / 4).  A lane holds of a block row
// lane % BLK, and columns 4 g .. 4 g + 3 (g = lane / 16) of 16, or 8 q + 4 g .. + 3
// (g = lane / 32) of 32.
template <int PASS, int MB, int NB, class ACC, class SLOT>
__device__ __forceinline__ void put_rows(v4f* mine, const ACC (&acc)[MB][NB], int pass,
                                         SLOT&& slot) {
  constexpr int Q = sizeof(ACC) / 16, BLK = Q == 1 ? 16 : 32;
  const int lane = threadIdx.x & 63, r = lane % BLK, g = lane / BLK;
#pragma unroll
  for (int i = 0; i < PASS / BLK; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const ACC& c = acc[pass * (PASS / BLK) + i][j];
      if constexpr (Q == 1) {
        mine[slot(i * BLK + r, 4 * j + g)] = c;
      } else {
#pragma unroll
        for (int q = 0; q < Q; ++q)
          mine[slot(i * BLK + r, 8 * j + 2 * q + g)] =
              v4f{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
      }
    }
}

// A wave's accumulators through its part of the LDS: each(row, column, eight columns'
// values, of(row)) for eight columns of a row at a time, the columns below N.  of() is what
// is read for a row: for all of a pass's rows at once, ahead of its stores, behind which
// the compiler would wait for each one.
template <class C, int LDS, int MB, int NB, class ACC, class OF, class EACH>
__device__ __forceinline__ void rows_through_lds(uint8_t* smem, const ACC (&acc)[MB][NB], int m0,
                                                 int n0, int M, int N, OF&& of, EACH&& each) {
  constexpr int PASS = C::pass_of(C::WTM, LDS);
  static_assert(PASS % (C::WTM / MB) == 0 && C::WTM % PASS == 0, "whole blocks per pass");
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wm = w / C::WGN, wn = w % C::WGN;
  constexpr int CH = C::WTN / 4, LPR = C::WTN / 8, RPI = 64 / LPR, TURNS = PASS / RPI;
  static_assert(RPI * LPR == 64 && TURNS * RPI == PASS, "whole turns");
  constexpr int SWZ = (CH & (CH - 1)) == 0 ? CH - 1 : 0;     // as tile_out
  auto slot = [](int r, int c) { return r * CH + (c ^ (r & SWZ)); };
  v4f* mine = reinterpret_cast<v4f*>(smem + w * (LDS / C::NW / 16 * 16));
  const int cl = lane % LPR, rl = lane / LPR;
  const int col = n0 + wn * C::WTN + cl * 8;
  const bool col_ok = col < N;                               // N is a multiple of 8
#pragma unroll
  for (int p = 0; p < C::WTM / PASS; ++p) {
    const int first = m0 + wm * C::WTM + p * PASS + rl;
    decltype(of(0)) info[TURNS];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) info[i] = of(min(first + i * RPI, M - 1));
    // the wave's own LDS: its accesses are executed in order
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    put_rows<PASS>(mine, acc, p, slot);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
      const int r = i * RPI + rl;
      const v4f a = mine[slot(r, 2 * cl)];
      const v4f b = mine[slot(r, 2 * cl + 1)];
      if (!col_ok || first + i * RPI >= M) continue;
      float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      each(first + i * RPI, col, v, info[i]);
    }
  }
}

// The epilogue of a wave's accumulators, through its part of the LDS.
template <class C, int LDS, class OT, bool STREAM, bool SPLIT, int MB, int NB, class ACC>
__device__ __forceinline__ void tile_out(uint8_t* smem, const ACC (&acc)[MB][NB], int m0, int n0,
                                         int M, int N, float scale, const Epilogue& ep,
                                         float* __restrict__ part, int sp) {
  constexpr int PASS = C::pass_of(C::WTM, LDS);
  static_assert(PASS % (C::WTM / MB) == 0 && C::WTM % PASS == 0, "whole blocks per pass");
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wm = w / C::WGN, wn = w % C::WGN;
  constexpr int CH = C::WTN / 4, LPR = C::WTN / 8, RPI = 64 / LPR;
  // 16-byte chunk c of row r: swizzled where the rows' stride is a power of two
  // (else the stride itself spreads the rows over the banks)
  constexpr int SWZ = (CH & (CH - 1)) == 0 ? CH - 1 : 0;
  auto slot = [](int r, int c) { return r * CH + (c ^ (r & SWZ)); };
  v4f* mine = reinterpret_cast<v4f*>(smem + w * (LDS / C::NW / 16 * 16));
  const int cl = lane % LPR, rl = lane / LPR;
  // A lane stores 16 bytes at a time, a row's lanes one run of them: eight columns of
  // bfloat16, or (RUNS) twice four of float32.  With a residual float32 is eight columns
  // side by side as well, and in the caches: a load waits for the stores ahead of it, and
  // the two runs have twice as many such waits, or lose more than those if both are read
  // ahead: 4096 x 4096 x 4096 63 us, 72 and 79 in runs; 4096 x 8192 x 4096 154, 182 and 210.
  constexpr bool F32 = SPLIT || sizeof(OT) == 4;
  const bool runs = F32 && (SPLIT || !ep.residual);
  const int c0 = runs ? cl : 2 * cl, c1 = runs ? cl + LPR : 2 * cl + 1;
  const int col0 = n0 + wn * C::WTN;
  const bool ok0 = rl < RPI && col0 + 4 * c0 < N;            // N is a multiple of 16
  const bool ok1 = rl < RPI && col0 + 4 * c1 < N;
  float b0[4], b1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b0[i] = b1[i] = 0.0f;
  if (!SPLIT && ep.bias) {
    if (ok0) load_elems<4>(ep.bias + col0 + 4 * c0, b0);
    if (ok1) load_elems<4>(ep.bias + col0 + 4 * c1, b1);
  }
  auto rows = [&](auto act, int first) {
    constexpr int ACT = decltype(act)::value;
    const auto run = [&](const v4f& a, const float (&bias)[4], int64_t at) {
      float v[4] = {a[0], a[1], a[2], a[3]};
      if constexpr (SPLIT)
        store_elems<4>(part + (int64_t)sp * M * N + at, v);
      else
        finish<ACT, OT, STREAM>(v, scale, bias, ep, at);
    };
    const auto side_by_side = [&](const v4f& a, const v4f& b, int64_t at) {
      float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      const float bias[8] = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
      finish<ACT, OT, STREAM && !F32>(v, scale, bias, ep, at);
    };
    const auto each_row = [&](auto in_runs) {
      for (int r = rl; r < PASS; r += RPI) {              // lanes past RPI rows: idle
        const int row = m0 + wm * C::WTM + first + r;
        const v4f a = mine[slot(r, c0)], b = mine[slot(r, c1)];
        const int64_t at = (int64_t)row * N + col0;
        if constexpr (decltype(in_runs)::value) {
          if (ok0 && row < M) run(a, b0, at + 4 * c0);
          if (ok1 && row < M) run(b, b1, at + 4 * c1);
        } else if constexpr (!SPLIT) {
          if (ok0 && row < M) side_by_side(a, b, at + 4 * c0);
        }
      }
    };
    if (runs)
      each_row(std::bool_constant<F32>{});
    else
      each_row(std::false_type{});
  };
#pragma unroll
  for (int p = 0; p < C::WTM / PASS; ++p) {
    // the wave's own LDS: its accesses are executed in order
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    put_rows<PASS>(mine, acc, p, slot);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int first = p * PASS;
    switch (SPLIT ? (int)kNone : ep.act) {
      case kRelu: rows(std::integral_constant<int, kRelu>{}, first); break;
      case kGelu: rows(std::integral_constant<int, kGelu>{}, first); break;
      case kGeluTanh: rows(std::integral_constant<int, kGeluTanh>{}, first); break;
      case kSilu: rows(std::integral_constant<int, kSilu>{}, first); break;
      default: rows(std::integral_constant<int, kNone>{}, first); break;
    }
  }
}

// LDS of tile_product: the stages (a step's rows of either operand; of a turned B the
// step's 64 rows of the tile's columns), then their exponent bytes, where there are any.
template <class OP, class C>
constexpr int kTileStage = OP::kTurned ? C::BM * C::BK + 64 * C::BN : C::STAGE;
template <class OP, class C>
constexpr int kTileLds = C::S * (kTileStage<OP, C> + (OP::kScaled ? (C::BM + C::BN) * 8 : 0));

// The tile at (m0, n0) over K steps k_lo .. steps - 1 (of all that K has): before()
// is called ahead of the loop, out(acc, what it gave, LDS) behind it, with the LDS
// (kTileLds) free.
template <class OP, class C, class BEFORE, class OUT>
__device__ __forceinline__ void tile_product(const uint8_t* __restrict__ A,
                                             const uint8_t* __restrict__ B, int M, int N, int K,
                                             int m0, int n0, int k_lo, int k_end,
                                             const Exponents& ex, BEFORE&& before, OUT&& out) {
  constexpr int BK = C::BK, MB = C::MB, NB = C::NB;
  // exponent bytes of a stage: 8 a row, a lane loads those of two rows
  constexpr int EROWS = C::BM + C::BN, ELANES = EROWS / 2 / C::NW;
  constexpr bool TURNED = OP::kTurned;
  constexpr int STAGE = kTileStage<OP, C>, BI = TURNED ? 64 * C::BN / 1024 / C::NW : C::BI;
  constexpr int LPS = C::AI + BI + OP::kScaled, CPR = C::BN / 16, RPL = 64 / CPR;
  static_assert(!TURNED || BI * C::NW * 1024 == 64 * C::BN, "whole loads");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kTileLds<OP, C>];
  static_assert(!OP::kScaled || (ELANES * 2 * C::NW == EROWS && ELANES <= 64), "whole rows");
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wm = w / C::WGN, wn = w % C::WGN;
  // the step at nk, if any, is the one of rem bytes
  // (turned: the one of fewer than 64 rows of B, whose columns of A are zeros)
  const int nk = TURNED ? ex.rows_b / 64 : K / BK, rem = TURNED ? 0 : K % BK;
  const int all = (K + BK - 1) / BK, steps = min(all, k_end);

  v4f acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;

  // per-lane source of each direct load: a row (clamped into the matrix) and
  // the swizzled chunk
  const int lrow = lane >> 3, lslot = lane & 7;
  const uint8_t* gA[C::AI];
  const uint8_t* gB[BI];
#pragma unroll
  for (int j = 0; j < C::AI; ++j) {
    const int row = (w * C::AI + j) * 8 + lrow;
    gA[j] = A + (int64_t)min(m0 + row, M - 1) * K + ((lslot ^ gemm::dma::swz(row)) * 16);
  }
  // turned: row lane / CPR of RPL, its chunk of columns clamped into the matrix
  const int trow = lane / CPR;
#pragma unroll
  for (int j = 0; j < BI; ++j) {
    if constexpr (TURNED) {
      const int row = (w * BI + j) * RPL + trow;
      const int chunk = (lane % CPR) ^ turned_swz<CPR>(row);
      gB[j] = B + (int64_t)row * N + min(n0 + chunk * 16, N - 16);
    } else {
      const int row = (w * BI + j) * 8 + lrow;
      gB[j] = B + (int64_t)min(n0 + row, N - 1) * K + ((lslot ^ gemm::dma::swz(row)) * 16);
    }
  }
  const uint8_t* gE = nullptr;
  int64_t estep = 0;
  if constexpr (OP::kScaled) {
    const int r = (w * ELANES + min(lane, ELANES - 1)) * 2;  // of A's rows, then B's
    const bool of_a = r < C::BM;
    const int rows = of_a ? ex.rows_a : ex.rows_b;           // multiples of 16
    gE = (of_a ? ex.a : ex.b) + (int64_t)min(of_a ? m0 + r : n0 + r - C::BM, rows - 2) * 8;
    estep = (int64_t)rows * 8;
  }
  auto issue_exponents = [&](int stage, int kt) {
    if constexpr (OP::kScaled)
      if (lane < ELANES)
        load16_to_lds(gE + kt * estep,
                      __builtin_amdgcn_readfirstlane(lds_offset(smem) + C::S * STAGE +
                                                     (stage * EROWS + w * ELANES * 2) * 8));
  };
  auto issue = [&](int stage, int k0) {
    const uint32_t base = lds_offset(smem + stage * STAGE);
    const uint32_t la = __builtin_amdgcn_readfirstlane(base + w * C::AI * 1024);
    const uint32_t lb = __builtin_amdgcn_readfirstlane(base + C::BM * BK + w * BI * 1024);
#pragma unroll
    for (int j = 0; j < C::AI; ++j) load16_to_lds(gA[j] + k0, la + j * 1024);
#pragma unroll
    for (int j = 0; j < BI; ++j) {
      int64_t at = k0;
      if constexpr (TURNED) {                                // rows past the last: the last
        const int row = (w * BI + j) * RPL + trow, first = k0 / 2;
        at = (int64_t)(first + min(0, ex.rows_b - 1 - first - row)) * N;
      }
      load16_to_lds(gB[j] + at, lb + j * 1024);
    }
  };
  // the step of fewer than BK bytes: chunks past K load the row's last chunk
  auto issue_rem = [&](int stage) {
    const uint32_t base = lds_offset(smem + stage * STAGE);
    const uint32_t la = __builtin_amdgcn_readfirstlane(base + w * C::AI * 1024);
    const uint32_t lb = __builtin_amdgcn_readfirstlane(base + C::BM * BK + w * BI * 1024);
#pragma unroll
    for (int j = 0; j < C::AI; ++j) {
      const int co = (lslot ^ gemm::dma::swz((w * C::AI + j) * 8 + lrow)) * 16;
      load16_to_lds(gA[j] + nk * BK - max(0, co - (rem - 16)), la + j * 1024);
    }
#pragma unroll
    for (int j = 0; j < BI; ++j) {
      const int co = (lslot ^ gemm::dma::swz((w * BI + j) * 8 + lrow)) * 16;
      load16_to_lds(gB[j] + nk * BK - max(0, co - (rem - 16)), lb + j * 1024);
    }
  };
  auto fetch = [&](int kt) {
    const int stage = (kt - k_lo) % C::S;
    if (TURNED || kt < nk)
      issue(stage, kt * BK);
    else
      issue_rem(stage);
    issue_exponents(stage, kt);
  };
#pragma unroll
  for (int s = 0; s < C::S - 1; ++s)
    if (k_lo + s < steps) fetch(k_lo + s);

  const int r16 = lane & 15, g = lane >> 4;
  const int sw = gemm::dma::swz(r16);
  const int o0 = (OP::chunk(g, 0) ^ sw) * 16, o1 = (OP::chunk(g, 1) ^ sw) * 16;
  const int offA = (wm * C::WTM + r16) * BK, offB = C::BM * BK + (wn * C::WTN + r16) * BK;
  // the fragment of the 16 rows from byte `at` of a stage on
  auto frag = [&](int stage, int at) {
    const uint8_t* p = smem + stage * STAGE + at;
    int e = 0;
    if constexpr (OP::kScaled)
      e = *reinterpret_cast<const typename OP::Scales*>(smem + C::S * STAGE +
                                                        stage * EROWS * 8 + at / BK * 8 + 2 * g);
    const uint4 q[2] = {*reinterpret_cast<const uint4*>(p + o0),
                        *reinterpret_cast<const uint4*>(p + o1)};
    return OP::make(q, e);
  };
  // of B, block j of the wave's columns
  int tB[NB];
  if constexpr (TURNED) {
    const int row = turned_row(lane);
#pragma unroll
    for (int j = 0; j < NB; ++j)
      tB[j] = C::BM * BK + (g * 8 + row) * C::BN + (lane & 1) * 8 +
              (((wn * C::WTN) / 16 + j) ^ turned_swz<CPR>(row)) * 16;
  }
  auto frag_b = [&](int stage, int j) {
    if constexpr (TURNED) {
      typename OP::FragB f;
#pragma unroll
      for (int p = 0; p < OP::kParts; ++p)
        f.h[p] = read_turned(smem + stage * STAGE + tB[j] + p * 32 * C::BN);
      return f;
    } else {
      return frag(stage, offB + j * 16 * BK);
    }
  };
  const auto kept = before();
  // fragment reads in the order the MFMAs consume them; next(): the loads of
  // the following stage, sent once the first fragments are in registers
  auto step = [&](int st, auto&& next) {
    typename OP::FragB bf[NB];
    typename OP::Frag af[2];
    af[0] = frag(st, offA);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      bf[j] = frag_b(st, j);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if (i + 1 < MB) af[(i + 1) & 1] = frag(st, offA + (i + 1) * 16 * BK);
      __builtin_amdgcn_sched_barrier(0);
      // D = B A^T per block: a lane ends with four columns of one row
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = OP::mma(bf[j], af[i & 1], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      if (i == 0) next();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  __builtin_amdgcn_s_waitcnt(0xC07F);                        // lgkmcnt(0)
  const int k_whole = TURNED ? steps : min(steps, nk);
  for (int kt = k_lo; kt < k_whole; ++kt) {
    wait_stages<C::S - 2, LPS>(steps - 1 - kt);
    barrier_no_drain();
    step((kt - k_lo) % C::S, [&] {
      if (kt + C::S - 1 < steps) fetch(kt + C::S - 1);
    });
  }
  if (rem && steps == all) {
    uint8_t* st = smem + (nk - k_lo) % C::S * STAGE;
    wait_vmem(0);
    barrier_no_drain();
    const int valid = rem / 16;                              // chunks of K in the step
    for (int i = tid; i < (C::BM + C::BN) * 8; i += C::kThreads) {
      const int row = i >> 3, c = i & 7;                     // BM is a multiple of 16
      if (c >= valid)
        *reinterpret_cast<uint4*>(st + row * BK + ((c ^ gemm::dma::swz(row & 15)) * 16)) =
            make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    step((nk - k_lo) % C::S, [] {});
  }
  __syncthreads();                                           // the stages are free
  out(acc, kept, smem);
}

// STREAM: the outputs go past the caches (kStreamOut in linear_act.hip).
// SPLIT (few tiles, long K): workgroup b takes tile b % tiles and the kc K steps
// of split b / tiles, and writes its sums, unscaled, to that split's plane of
// `part` ([M x N] floats each); linear_act_join adds the planes in order.
template <class OP, class C, class OT, bool STREAM, bool SPLIT = false>
__global__ __launch_bounds__(C::kThreads) void linear_act_tile(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, Epilogue ep, Exponents ex, float* __restrict__ part = nullptr, int kc = 0) {
  int tm, tn;
  const int nt = tilesM * tilesN, sp = SPLIT ? (int)blockIdx.x / nt : 0;
  gemm::tile_of(gemm::xcd_remap((int)blockIdx.x - sp * nt, nt), tilesM, tilesN, tm, tn);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  tile_product<OP, C>(
      A, B, M, N, K, m0, n0, SPLIT ? sp * kc : 0, SPLIT ? sp * kc + kc : INT32_MAX, ex,
      [&] { return scale_of<OP>(ep); },
      [&](const v4f (&acc)[C::MB][C::NB], float scale, uint8_t* smem) {
        tile_out<C, kTileLds<OP, C>, OT, STREAM, SPLIT>(smem, acc, m0, n0, M, N, scale, ep, part,
                                                        sp);
      });
}

// y (and z) from the S planes of partial sums
template <int ACT, class OT>
__device__ __forceinline__ void join8(const float* __restrict__ part, int S, int64_t plane,
                                      int64_t at, int col, float scale, const Epilogue& ep) {
  float v[8], bias[8];
  load_elems<8>(part + at, v);
  for (int s = 1; s < S; ++s) {
    float t[8];
    load_elems<8>(part + s * plane + at, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = 0.0f;
  if (ep.bias) load_elems<8>(ep.bias + col, bias);
  finish<ACT, OT, false>(v, scale, bias, ep, at);
}
template <class OP, class OT>
__global__ __launch_bounds__(256) void linear_act_join(const float* __restrict__ part, int S,
                                                       int64_t M, int N, Epilogue ep) {
  const int64_t plane = M * N;
  const float scale = scale_of<OP>(ep);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < plane / 8;
       i += (int64_t)gridDim.x * 256) {
    const int64_t at = i * 8;
    const int col = (int)(at % N);
    switch (ep.act) {
      case kRelu: join8<kRelu, OT>(part, S, plane, at, col, scale, ep); break;
      case kGelu: join8<kGelu, OT>(part, S, plane, at, col, scale, ep); break;
      case kGeluTanh: join8<kGeluTanh, OT>(part, S, plane, at, col, scale, ep); break;
      case kSilu: join8<kSilu, OT>(part, S, plane, at, col, scale, ep); break;
      default: join8<kNone, OT>(part, S, plane, at, col, scale, ep); break;
    }
  }
}

}  // namespace
}  // namespace falq
