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

// The epilogue of a wave's accumulators, through its part of the LDS.
template <class C, int LDS, class OT, bool STREAM, bool SPLIT>
__device__ __forceinline__ void tile_out(uint8_t* smem, const v4f (&acc)[C::MB][C::NB], int m0,
                                         int n0, int M, int N, float scale, const Epilogue& ep,
                                         float* __restrict__ part, int sp) {
  constexpr int NB = C::NB, PASS = C::pass_of(C::WTM, LDS);
  static_assert(PASS % 16 == 0 && C::WTM % PASS == 0, "whole blocks per pass");
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wm = w / C::WGN, wn = w % C::WGN;
  const int r16 = lane & 15, g = lane >> 4;
  constexpr int CH = C::WTN / 4, LPR = C::WTN / 8, RPI = 64 / LPR;
  // 16-byte chunk c of row r: swizzled where the rows' stride is a power of two
  // (else the stride itself spreads the rows over the banks)
  constexpr int SWZ = (CH & (CH - 1)) == 0 ? CH - 1 : 0;
  auto slot = [](int r, int c) { return r * CH + (c ^ (r & SWZ)); };
  v4f* mine = reinterpret_cast<v4f*>(smem + w * (LDS / C::NW / 16 * 16));
  const int cl = lane % LPR, rl = lane / LPR;
  const int col = n0 + wn * C::WTN + cl * 8;
  const bool col_ok = rl < RPI && col < N;                   // N is a multiple of 16
  float bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = 0.0f;
  if (!SPLIT && ep.bias && col_ok) load_elems<8>(ep.bias + col, bias);
  auto rows = [&](auto act, int first) {
    for (int r = rl; r < PASS; r += RPI) {                // lanes past RPI rows: idle
      const int row = m0 + wm * C::WTM + first + r;
      const v4f a = mine[slot(r, 2 * cl)];
      const v4f b = mine[slot(r, 2 * cl + 1)];
      if (!col_ok || row >= M) continue;
      float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      if constexpr (SPLIT)
        store_elems<8>(part + ((int64_t)sp * M + row) * N + col, v);
      else
        finish8<decltype(act)::value, OT, STREAM>(v, scale, bias, ep, (int64_t)row * N + col);
    }
  };
#pragma unroll
  for (int p = 0; p < C::WTM / PASS; ++p) {
    // the wave's own LDS: its accesses are executed in order
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < PASS / 16; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        mine[slot(i * 16 + r16, 4 * j + g)] = acc[p * (PASS / 16) + i][j];
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

// STREAM: the outputs go past the caches (kStreamOut in linear_act.hip).
// SPLIT (few tiles, long K): workgroup b takes tile b % tiles and the kc K steps
// of split b / tiles, and writes its sums, unscaled, to that split's plane of
// `part` ([M x N] floats each); linear_act_join adds the planes in order.
template <class C, class OT, bool STREAM, bool SPLIT = false>
__global__ __launch_bounds__(C::kThreads) void linear_act_tile(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, Epilogue ep, float* __restrict__ part = nullptr, int kc = 0) {
  constexpr int BK = C::BK, MB = C::MB, NB = C::NB;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::S * C::STAGE];
  int tm, tn;
  const int nt = tilesM * tilesN, sp = SPLIT ? (int)blockIdx.x / nt : 0;
  gemm::tile_of(gemm::xcd_remap((int)blockIdx.x - sp * nt, nt), tilesM, tilesN, tm, tn);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wm = w / C::WGN, wn = w % C::WGN;
  // the step at nk, if any, is the one of rem bytes
  const int nk = K / BK, rem = K % BK, all = nk + (rem > 0);
  const int k_lo = SPLIT ? sp * kc : 0, steps = SPLIT ? min(all, k_lo + kc) : all;

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
  const uint8_t* gB[C::BI];
#pragma unroll
  for (int j = 0; j < C::AI; ++j) {
    const int row = (w * C::AI + j) * 8 + lrow;
    gA[j] = A + (int64_t)min(m0 + row, M - 1) * K + ((lslot ^ gemm::dma::swz(row)) * 16);
  }
#pragma unroll
  for (int j = 0; j < C::BI; ++j) {
    const int row = (w * C::BI + j) * 8 + lrow;
    gB[j] = B + (int64_t)min(n0 + row, N - 1) * K + ((lslot ^ gemm::dma::swz(row)) * 16);
  }
  auto issue = [&](int stage, int k0) {
    const uint32_t base = lds_offset(smem + stage * C::STAGE);
    const uint32_t la = __builtin_amdgcn_readfirstlane(base + w * C::AI * 1024);
    const uint32_t lb = __builtin_amdgcn_readfirstlane(base + C::BM * BK + w * C::BI * 1024);
#pragma unroll
    for (int j = 0; j < C::AI; ++j) load16_to_lds(gA[j] + k0, la + j * 1024);
#pragma unroll
    for (int j = 0; j < C::BI; ++j) load16_to_lds(gB[j] + k0, lb + j * 1024);
  };
  // the step of fewer than BK bytes: chunks past K load the row's last chunk
  auto issue_rem = [&](int stage) {
    const uint32_t base = lds_offset(smem + stage * C::STAGE);
    const uint32_t la = __builtin_amdgcn_readfirstlane(base + w * C::AI * 1024);
    const uint32_t lb = __builtin_amdgcn_readfirstlane(base + C::BM * BK + w * C::BI * 1024);
#pragma unroll
    for (int j = 0; j < C::AI; ++j) {
      const int co = (lslot ^ gemm::dma::swz((w * C::AI + j) * 8 + lrow)) * 16;
      load16_to_lds(gA[j] + nk * BK - max(0, co - (rem - 16)), la + j * 1024);
    }
#pragma unroll
    for (int j = 0; j < C::BI; ++j) {
      const int co = (lslot ^ gemm::dma::swz((w * C::BI + j) * 8 + lrow)) * 16;
      load16_to_lds(gB[j] + nk * BK - max(0, co - (rem - 16)), lb + j * 1024);
    }
  };
  auto fetch = [&](int kt) {
    const int stage = (kt - k_lo) % C::S;
    if (kt < nk)
      issue(stage, kt * BK);
    else
      issue_rem(stage);
  };
#pragma unroll
  for (int s = 0; s < C::S - 1; ++s)
    if (k_lo + s < steps) fetch(k_lo + s);

  const int r16 = lane & 15, g = lane >> 4;
  const int sw = gemm::dma::swz(r16);
  const int o0 = ((2 * g) ^ sw) * 16, o1 = ((2 * g + 1) ^ sw) * 16;
  const int offA = (wm * C::WTM + r16) * BK, offB = C::BM * BK + (wn * C::WTN + r16) * BK;
  auto frag = [&](const uint8_t* p) {
    return gemm::join(*reinterpret_cast<const uint4*>(p + o0),
                      *reinterpret_cast<const uint4*>(p + o1));
  };
  const float scale = 1.0f / (ep.sa[0] * ep.sb[0]);
  // fragment reads in the order the MFMAs consume them; next(): the loads of
  // the following stage, sent once the first fragments are in registers
  auto step = [&](const uint8_t* st, auto&& next) {
    v8i bf[NB], af[2];
    af[0] = frag(st + offA);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      bf[j] = frag(st + offB + j * 16 * BK);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      if (i + 1 < MB) af[(i + 1) & 1] = frag(st + offA + (i + 1) * 16 * BK);
      __builtin_amdgcn_sched_barrier(0);
      // D = B A^T per block: a lane ends with four columns of one row
#pragma unroll
      for (int j = 0; j < NB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af[i & 1], acc[i][j],
                                                                     0, 0, 0, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (i == 0) next();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  __builtin_amdgcn_s_waitcnt(0xC07F);                        // lgkmcnt(0)
  const int k_whole = min(steps, nk);
  for (int kt = k_lo; kt < k_whole; ++kt) {
    wait_stages<C::S - 2, C::LPS>(steps - 1 - kt);
    barrier_no_drain();
    step(smem + (kt - k_lo) % C::S * C::STAGE, [&] {
      if (kt + C::S - 1 < steps) fetch(kt + C::S - 1);
    });
  }
  if (rem && steps == all) {
    uint8_t* st = smem + (nk - k_lo) % C::S * C::STAGE;
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
    step(st, [] {});
  }
  __syncthreads();                                           // the stages are free

  tile_out<C, C::S * C::STAGE, OT, STREAM, SPLIT>(smem, acc, m0, n0, M, N, scale, ep, part, sp);
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
  finish8<ACT, OT, false>(v, scale, bias, ep, at);
}
template <class OT>
__global__ __launch_bounds__(256) void linear_act_join(const float* __restrict__ part, int S,
                                                       int64_t M, int N, Epilogue ep) {
  const int64_t plane = M * N;
  const float scale = 1.0f / (ep.sa[0] * ep.sb[0]);
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
