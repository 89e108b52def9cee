// The FP8 product of a melded linear layer with its epilogue:
//   z = dec(X~) dec(W~)^T / (s_x s_w) + bias,   y = act(z) + residual,
// y, z and residual all bfloat16 or all float32; z is written where the
// caller keeps it for the backward.  Accumulation, bias, activation and
// residual are float32, and each output is rounded once.
//
// Tiles: the scheme of the direct-to-LDS kernel in gemm_fp8_kernel.hpp (two
// LDS stages of 128 K-bytes, v_mfma_f32_16x16x128_f8f6f4, XOR-swizzled rows),
// for any tile size and any K that is a multiple of 16: in a last step of
// fewer than 128 bytes the chunks past K are cleared in LDS.
//
// Epilogue: a lane holds four columns of a row per 16 x 16 block, so a store
// from the registers would be 8 or 16 bytes wide.  Each wave passes its
// accumulators through its own part of the LDS (16-byte chunks XOR-swizzled
// by the row: no bank conflicts either way) and reads them back as eight
// columns of a row per lane; bias, residual and the outputs are then 16-byte
// accesses on whole 128-byte lines, and the epilogue's code is a short loop
// instead of one copy per accumulator.
#include "activation.hpp"
#include "elem.hpp"
#include "gemm_fp8_kernel.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace falq {
namespace {

struct Epilogue {
  const float* sa;
  const float* sb;
  const float* bias;        // [N] or null
  const void* residual;     // [M x N] or null; may be y
  void* y;                  // [M x N]
  void* z;                  // [M x N] or null
  int act;
};

// eight columns of one row
template <int ACT, class OT>
__device__ __forceinline__ void finish8(float (&v)[8], float scale, const float (&bias)[8],
                                        const Epilogue& e, int64_t at) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], scale, bias[i]);
  if (e.z) store_elems<8>((OT*)e.z + at, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = act_value<ACT>(v[i]);
  if (e.residual) {
    float r[8];
    load_elems<8>((const OT*)e.residual + at, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  store_elems<8>((OT*)e.y + at, v);
}

template <int BM_, int BN_, int WGM_, int WGN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, BK = 128, S = 2;
  static constexpr int NW = WGM * WGN, kThreads = NW * 64;
  static constexpr int WTM = BM / WGM, WTN = BN / WGN, MB = WTM / 16, NB = WTN / 16;
  static constexpr int STAGE = (BM + BN) * BK;
  static constexpr int AI = BM / 8 / NW, BI = BN / 8 / NW;   // 1 KB loads per wave and stage
  // the epilogue: rows of a wave's sub-tile per pass through its LDS
  static constexpr int PASS = S * STAGE / NW / (WTN * 4) < WTM ? S * STAGE / NW / (WTN * 4) : WTM;
  static_assert(AI * 8 * NW == BM && BI * 8 * NW == BN, "whole loads");
  static_assert(S * STAGE <= 160 * 1024, "LDS");
  static_assert(PASS % 16 == 0 && WTM % PASS == 0, "whole blocks per pass");
};

template <class C, class OT>
__global__ __launch_bounds__(C::kThreads) void linear_act_tile(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int n_first,
    int tilesM, int tilesN, Epilogue ep) {
  constexpr int BK = C::BK, MB = C::MB, NB = C::NB;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::S * C::STAGE];
  int tm, tn;
  gemm::tile_of(gemm::xcd_remap(blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = tm * C::BM, n0 = n_first + tn * C::BN;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wm = w / C::WGN, wn = w % C::WGN;
  const int nk = K / BK, rem = K % BK;

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
  if (nk > 0)
    issue(0, 0);
  else if (rem)
    issue_rem(0);

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
  for (int kt = 0; kt < nk; ++kt) {
    wait_vmem(0);
    barrier_no_drain();
    step(smem + (kt & 1) * C::STAGE, [&] {
      if (kt + 1 < nk)
        issue((kt + 1) & 1, (kt + 1) * BK);
      else if (rem)
        issue_rem((kt + 1) & 1);
    });
  }
  if (rem) {
    uint8_t* st = smem + (nk & 1) * C::STAGE;
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

  constexpr int CH = C::WTN / 4, LPR = C::WTN / 8, RPI = 64 / LPR;
  v4f* mine = reinterpret_cast<v4f*>(smem + w * (C::S * C::STAGE / C::NW));
  const int cl = lane % LPR, rl = lane / LPR;
  const int col = n0 + wn * C::WTN + cl * 8;
  const bool col_ok = col < N;                               // N is a multiple of 16
  float bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = 0.0f;
  if (ep.bias && col_ok) load_elems<8>(ep.bias + col, bias);
  auto rows = [&](auto act, int first) {
    for (int r = rl; r < C::PASS; r += RPI) {
      const int row = m0 + wm * C::WTM + first + r;
      const v4f a = mine[r * CH + ((2 * cl) ^ (r & (CH - 1)))];
      const v4f b = mine[r * CH + ((2 * cl + 1) ^ (r & (CH - 1)))];
      if (!col_ok || row >= M) continue;
      float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      finish8<decltype(act)::value, OT>(v, scale, bias, ep, (int64_t)row * N + col);
    }
  };
#pragma unroll
  for (int p = 0; p < C::WTM / C::PASS; ++p) {
    // the wave's own LDS: its accesses are executed in order
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < C::PASS / 16; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        mine[(i * 16 + r16) * CH + ((4 * j + g) ^ ((i * 16 + r16) & (CH - 1)))] =
            acc[p * (C::PASS / 16) + i][j];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int first = p * C::PASS;
    switch (ep.act) {
      case kRelu: rows(std::integral_constant<int, kRelu>{}, first); break;
      case kGelu: rows(std::integral_constant<int, kGelu>{}, first); break;
      case kGeluTanh: rows(std::integral_constant<int, kGeluTanh>{}, first); break;
      case kSilu: rows(std::integral_constant<int, kSilu>{}, first); break;
      default: rows(std::integral_constant<int, kNone>{}, first); break;
    }
  }
}

// output columns [n_first, n_end) in tiles of C
template <class C, class OT>
hipError_t launch_tiles(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                        int64_t n_first, int64_t n_end, const Epilogue& ep, hipStream_t s) {
  const int tM = (int)((M + C::BM - 1) / C::BM);
  const int tN = (int)((n_end - n_first + C::BN - 1) / C::BN);
  linear_act_tile<C, OT><<<tM * tN, C::kThreads, 0, s>>>(A, B, (int)M, (int)N, (int)K,
                                                         (int)n_first, tM, tN, ep);
  return hipGetLastError();
}

template <class OT>
hipError_t by_size(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                   const Epilogue& ep, hipStream_t s) {
  const auto tiles = [&](int64_t b) { return ((M + b - 1) / b) * ((N + b - 1) / b); };
  if (tiles(256) >= 128) return launch_tiles<Tile<256, 256, 2, 4>, OT>(A, B, M, N, K, 0, N, ep, s);
  if (tiles(128) >= 128) return launch_tiles<Tile<128, 128, 2, 2>, OT>(A, B, M, N, K, 0, N, ep, s);
  return launch_tiles<Tile<64, 64, 2, 2>, OT>(A, B, M, N, K, 0, N, ep, s);
}

}  // namespace

hipError_t launch_linear_act(const uint8_t* xq, const float* s_x, const uint8_t* wq,
                             const float* s_w, const float* bias, const void* residual, int64_t T,
                             int64_t d_in, int64_t d_out, int act, int dtype, void* y, void* z,
                             hipStream_t s) {
  if (T == 0 || d_out == 0) return hipSuccess;
  const Epilogue ep{s_x, s_w, bias, residual, y, z, act};
  return dtype == 0 ? by_size<float>(xq, wq, T, d_out, d_in, ep, s)
                    : by_size<__bf16>(xq, wq, T, d_out, d_in, ep, s);
}

}  // namespace falq
