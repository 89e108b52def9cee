// The FP8 product of a melded linear layer with its epilogue:
//   z = dec(X~) dec(W~)^T / (s_x s_w) + bias,   y = act(z) + residual,
// y, z and residual all bfloat16 or all float32; z is written where the
// caller keeps it for the backward.  Accumulation, bias, activation and
// residual are float32, and each output is rounded once.
//
// Tiles: the scheme of the direct-to-LDS kernel in gemm_fp8_kernel.hpp (two
// to four LDS stages of 128 K-bytes, v_mfma_f32_16x16x128_f8f6f4, swizzled rows),
// for any tile size and any K that is a multiple of 16: in a last step of
// fewer than 128 bytes the chunks past K are cleared in LDS.
//
// Long products are bound by the matrix cores (8192 x 11008 x 4096 with gelu and
// z: 329 us, 2.2 PFLOP/s; 280 without the epilogue's work and stores; 4096 x 5120
// x 13824 with a residual 228 us, 2.5 PFLOP/s), few tokens by reading W~ (1 x 4096
// x 4096: 5.2 us on the GPU, 3.2 TB/s, of which a launch's latency is half).
// Workgroups that keep their CU over several tiles, the next tile's first loads
// under the last K step and the stores draining under the next tile, measured no
// faster (354 us against 348 in one kind of tile): the long products run at the
// card's power limit.
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
  const int64_t out = M * N * (int64_t)sizeof(OT) *
                      (1 + (ep.z != nullptr) + (ep.residual != nullptr));
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

// Which tile: the one whose rounds of the 256 CUs take least.  A K step of a
// round of tiles costs (us, measured at 256 to 1024 tiles and 4096 and 8192
// K-bytes)
//     256 x 320  2.1      256 x 256  1.68     256 x 128  1.08     128 x 256  1.08
//     192 x 128  0.82     128 x 192  0.82     128 x 128  0.62
//      64 x  64  0.27      32 x  64  0.24
// and a launch about 4 more for the first loads and the last stores: a larger
// tile moves fewer bytes per product but leaves more of its last round empty.
// 512 x 4096 x 4096: 15.5 in tiles of 64 x 64, 18.9 in 128 x 128 (half a round),
// 17.5 in 32 x 128; 128 x 4096: 10.0 in 32 x 64, 10.9 in 64 x 64, 14 in 64 x
// 128; 4096 x 5120 x 13824: 230 in 256 x 320 (one round), 252 in
// a round of 256 x 256 and one of 128 x 128, 345 in 256 x 256; 512 x 11008 x 4096
// with gelu and z: 31.5 in 128 x 192 (232 tiles), 36.7 in 128 x 256, 45 in 128 x
// 128.
enum TileKind {
  k256, k256x320, k256x128, k128x256, k192x128, k128x192, k128, k64, k32x64, kTileKinds
};
constexpr int kTileM[kTileKinds] = {256, 256, 256, 128, 192, 128, 128, 64, 32};
constexpr int kTileN[kTileKinds] = {256, 320, 128, 256, 128, 192, 128, 64, 64};
constexpr float kStep[kTileKinds] = {1.68f, 2.1f,  1.08f, 1.08f, 0.82f,
                                     0.82f, 0.62f, 0.27f, 0.24f};
constexpr float kLaunch = 4.0f;
constexpr int kCUs = 256;

int64_t tiles_of(TileKind k, int64_t M, int64_t n) {
  return ((M + kTileM[k] - 1) / kTileM[k]) * ((n + kTileN[k] - 1) / kTileN[k]);
}

float tile_cost(TileKind k, int64_t M, int64_t n, int64_t steps) {
  const int64_t nt = tiles_of(k, M, n);
  // a grid holds fewer than 2^32 threads: very long outputs take large tiles
  if (k != k256 && nt >= 1 << 23) return HUGE_VALF;
  return kLaunch + kStep[k] * (float)steps * (float)((nt + kCUs - 1) / kCUs);
}

TileKind best_tile(int64_t M, int64_t n, int64_t steps) {
  int best = 0;
  for (int k = 1; k < kTileKinds; ++k)
    if (tile_cost((TileKind)k, M, n, steps) < tile_cost((TileKind)best, M, n, steps)) best = k;
  return (TileKind)best;
}

// How a product runs: by few tokens, by tiles of one kind, by whole rounds of
// 256 x 256 tiles (cols of their columns) and the remaining columns in tiles of
// `kind`, or by 128 x 128 tiles split over K (`split` parts, kc steps each).
struct Plan {
  int few = 0;
  TileKind kind = k256;
  int64_t cols = 0;
  int split = 1, kc = 0;
};

Plan plan_of(int64_t M, int64_t N, int64_t K) {
  Plan p;
  const int64_t steps = (K + 127) / 128;
  // few tokens: 4096 x 4096 5.6 us at 1 token and 6.6 at 16 (tiles of 32 x 64:
  // 9.5); at 32 tokens 8.3 against 9.6 while one workgroup per CU holds all
  // columns, 21 against 14.4 at 11008 columns
  if (K > 0 && M <= 16) p.few = 1;
  if (K > 0 && M > 16 && M <= 32 && N <= 16 * kCUs) p.few = 2;
  if (p.few) return p;
  p.kind = best_tile(M, N, steps);
  float cost = tile_cost(p.kind, M, N, steps);
  // whole rounds of large tiles, and the columns of a short last round in
  // smaller ones by a second launch
  const int64_t tM = (M + 255) / 256, tN = (N + 255) / 256;
  const int64_t c = tM * tN / kCUs * kCUs / tM;              // tile columns in whole rounds
  if (c > 0 && c < tN) {
    const TileKind k2 = best_tile(M, N - c * 256, steps);
    const float both = tile_cost(k256, M, c * 256, steps) + tile_cost(k2, M, N - c * 256, steps);
    if (both < cost) {
      cost = both;
      p.kind = k2;
      p.cols = c * 256;
    }
  }
  // few tiles and a long K: as many splits as give a workgroup to each CU, at
  // least 8 steps each, and the planes written and read once at 4 TB/s.  64 x
  // 5120 x 13824: 22.5 us in 6 splits, 32.5 whole; 100 x 4096 x 11008: 19.8 in
  // 8, 25.8 whole; 512 x 4096 x 4096 21.1 in 2, 15.5 whole.
  const int64_t nt = tiles_of(k128, M, N);
  const int64_t s = nt > 0 ? std::min<int64_t>(kCUs / nt, steps / 8) : 0;
  if (s >= 2) {
    const int64_t kc = (steps + s - 1) / s, parts = (steps + kc - 1) / kc;
    const float split = 2 * kLaunch + kStep[k128] * (float)kc +
                        (float)(parts * M * N) * 8.0f / 4e6f;
    if (parts >= 2 && split < cost) {
      p.kind = k128;
      p.cols = 0;
      p.split = (int)parts;
      p.kc = (int)kc;
    }
  }
  return p;
}

template <class OT>
hipError_t launch_kind(TileKind k, const uint8_t* A, const uint8_t* B, int64_t M, int64_t N,
                       int64_t K, int64_t n_first, int64_t n_end, const Epilogue& ep,
                       hipStream_t s) {
  switch (k) {
    case k256: return launch_tiles<Tile<256, 256, 2, 4>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k256x320:
      return launch_tiles<Tile<256, 320, 2, 4>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k256x128:
      return launch_tiles<Tile<256, 128, 4, 2, 3>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k192x128:
      return launch_tiles<Tile<192, 128, 2, 4, 3>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k128x192:
      return launch_tiles<Tile<128, 192, 2, 4, 3>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k128x256:
      return launch_tiles<Tile<128, 256, 2, 4, 3>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k128:
      return launch_tiles<Tile<128, 128, 2, 4, 3>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    case k64: return launch_tiles<Tile<64, 64, 2, 2, 4>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
    default: return launch_tiles<Tile<32, 64, 1, 4, 4>, OT>(A, B, M, N, K, n_first, n_end, ep, s);
  }
}

template <class OT>
hipError_t launch_split(const Plan& p, const uint8_t* A, const uint8_t* B, int64_t M, int64_t N,
                        int64_t K, const Epilogue& ep, float* part, hipStream_t s) {
  using C = Tile<128, 128, 2, 4, 3>;
  const int tM = (int)((M + C::BM - 1) / C::BM), tN = (int)((N + C::BN - 1) / C::BN);
  linear_act_tile<C, OT, false, true><<<tM * tN * p.split, C::kThreads, 0, s>>>(
      A, B, (int)M, (int)N, (int)K, 0, tM, tN, ep, part, p.kc);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int blocks = (int)std::min<int64_t>((M * N / 8 + 255) / 256, 2048);
  linear_act_join<OT><<<blocks, 256, 0, s>>>(part, p.split, M, (int)N, ep);
  return hipGetLastError();
}

template <class OT>
hipError_t by_plan(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                   const Epilogue& ep, float* part, hipStream_t s) {
  const Plan p = plan_of(M, N, K);
  if (p.few == 1) return launch_few<1, 1, 16, 1, OT>(A, B, M, N, K, ep, s);
  if (p.few == 2) return launch_few<2, 1, 8, 2, OT>(A, B, M, N, K, ep, s);
  if (p.split > 1) return launch_split<OT>(p, A, B, M, N, K, ep, part, s);
  if (p.cols > 0) {
    const hipError_t e = launch_kind<OT>(k256, A, B, M, N, K, 0, p.cols, ep, s);
    if (e != hipSuccess) return e;
  }
  return launch_kind<OT>(p.kind, A, B, M, N, K, p.cols, N, ep, s);
}

}  // namespace

size_t linear_act_ws_bytes(int64_t T, int64_t d_in, int64_t d_out) {
  if (T == 0 || d_out == 0) return 0;
  const Plan p = plan_of(T, d_out, d_in);
  return p.split > 1 ? (size_t)p.split * (size_t)T * (size_t)d_out * 4 : 0;
}

hipError_t launch_linear_act(const uint8_t* xq, const float* s_x, const uint8_t* wq,
                             const float* s_w, const float* bias, const void* residual, int64_t T,
                             int64_t d_in, int64_t d_out, int act, int dtype, void* y, void* z,
                             void* ws, hipStream_t s) {
  if (T == 0 || d_out == 0) return hipSuccess;
  const Epilogue ep{s_x, s_w, bias, residual, y, z, act};
  return dtype == 0 ? by_plan<float>(xq, wq, T, d_out, d_in, ep, (float*)ws, s)
                    : by_plan<__bf16>(xq, wq, T, d_out, d_in, ep, (float*)ws, s);
}

}  // namespace falq
