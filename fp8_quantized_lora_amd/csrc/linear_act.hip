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
#include "linear_act_tile.hpp"

#include <algorithm>
#include <cmath>

namespace falq {
namespace {

// output columns [n_first, n_end) in tiles of C
template <class C, class OT>
hipError_t launch_tiles(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                        int64_t n_first, int64_t n_end, const Epilogue& ep, hipStream_t s) {
  const int tM = (int)((M + C::BM - 1) / C::BM);
  const int tN = (int)((n_end - n_first + C::BN - 1) / C::BN);
  const int64_t out = M * N * (int64_t)sizeof(OT) * (1 + (ep.z != nullptr) + (ep.residual != nullptr));
  // the streaming hint needs whole lines: 16-byte stores, so bfloat16
  if (sizeof(OT) == 2 && out + M * K + N * K > kStreamBytes)
    linear_act_tile<C, OT, sizeof(OT) == 2><<<tM * tN, C::kThreads, 0, s>>>(
        A, B, (int)M, (int)N, (int)K, (int)n_first, tM, tN, ep);
  else
    linear_act_tile<C, OT, false><<<tM * tN, C::kThreads, 0, s>>>(
        A, B, (int)M, (int)N, (int)K, (int)n_first, tM, tN, ep);
  return hipGetLastError();
}

template <int MT, int NB, int NW, int U, class OT>
hipError_t launch_few(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                      const Epilogue& ep, hipStream_t s) {
  linear_act_few<MT, NB, NW, U, OT><<<(int)((N + NB * 16 - 1) / (NB * 16)), NW * 64, 0, s>>>(
      A, B, (int)M, (int)N, (int)K, ep);
  return hipGetLastError();
}

// Which tile: the one whose rounds of the 256 CUs take least.  A round of
// tiles costs, at 4096 K-bytes (us, measured at 256, 512, 768 and 1024 tiles;
// 5 more for the first loads and the last stores, whatever the tile):
//     256 x 320   75     256 x 256   58     128 x 128   20
//      64 x 128   11      64 x  64    7      32 x  64    5.6
// so a larger tile moves fewer bytes per product but leaves more of its last
// round empty.  512 x 4096 outputs: 15.3 in tiles of 64 x 128 (one round), 18.9
// in 128 x 128 (half a round), 17.5 in 32 x 128; 128 x 4096: 10.0 in 32 x 64,
// 10.9 in 64 x 64, 14 in 64 x 128.
enum TileKind { k256, k256x320, k128, k64x128, k64, k32x64, kTileKinds };
constexpr int kTileM[kTileKinds] = {256, 256, 128, 64, 64, 32};
constexpr int kTileN[kTileKinds] = {256, 320, 128, 128, 64, 64};
constexpr float kRound[kTileKinds] = {58.0f, 75.0f, 20.0f, 11.0f, 7.0f, 5.6f};
constexpr int kCUs = 256;

float tile_cost(TileKind k, int64_t M, int64_t n) {
  const int64_t nt = ((M + kTileM[k] - 1) / kTileM[k]) * ((n + kTileN[k] - 1) / kTileN[k]);
  // a grid holds fewer than 2^32 threads: very long outputs take large tiles
  if (k != k256 && nt >= 1 << 23) return HUGE_VALF;
  return kRound[k] * (float)((nt + kCUs - 1) / kCUs);
}

TileKind best_tile(int64_t M, int64_t n) {
  int best = 0;
  for (int k = 1; k < kTileKinds; ++k)
    if (tile_cost((TileKind)k, M, n) < tile_cost((TileKind)best, M, n)) best = k;
  return (TileKind)best;
}

template <class OT>
hipError_t launch_kind(TileKind k, const uint8_t* A, const uint8_t* B, int64_t M, int64_t N,
                       int64_t K, int64_t n_first, int64_t n_end, const Epilogue& ep,
                       hipStream_t s) {
  switch (k) {
    case k256: return launch_tiles<Tile<256, 256, 2, 4>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k256x320:
      return launch_tiles<Tile<256, 320, 2, 4>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k128:
      return launch_tiles<Tile<128, 128, 2, 4, 3>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k64x128:
      return launch_tiles<Tile<64, 128, 2, 4, 3>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k64: return launch_tiles<Tile<64, 64, 2, 2, 4>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    default: return launch_tiles<Tile<32, 64, 1, 4, 4>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
  }
}

template <class OT>
hipError_t by_size(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                   const Epilogue& ep, hipStream_t s) {
  // few tokens: 4096 x 4096 5.6 us at 1 token and 6.6 at 16 (tiles of 32 x 64:
  // 9.5); at 32 tokens 8.3 against 9.6 while one workgroup per CU holds all
  // columns, 21 against 14.4 at 11008 columns
  if (K > 0 && M <= 16) return launch_few<1, 1, 16, 1, OT>(A, B, M, N, K, ep, s);
  if (K > 0 && M <= 32 && N <= 16 * kCUs) return launch_few<2, 1, 8, 2, OT>(A, B, M, N, K, ep, s);
  const TileKind k = best_tile(M, N);
  // whole rounds of large tiles, and the columns of a short last round in
  // smaller ones (a second launch, about 3 us)
  const int64_t tM = (M + 255) / 256, tN = (N + 255) / 256;
  const int64_t c = tM * tN / kCUs * kCUs / tM;              // tile columns in whole rounds
  if (c > 0 && c < tN) {
    const TileKind k2 = best_tile(M, N - c * 256);
    if (tile_cost(k256, M, c * 256) + tile_cost(k2, M, N - c * 256) + 3.0f < tile_cost(k, M, N)) {
      const hipError_t e = launch_kind<OT>(k256, A, B, M, N, K, 0, c * 256, ep, s);
      if (e != hipSuccess) return e;
      return launch_kind<OT>(k2, A, B, M, N, K, c * 256, N, ep, s);
    }
  }
  return launch_kind<OT>(k, A, B, M, N, K, 0, N, ep, s);
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
