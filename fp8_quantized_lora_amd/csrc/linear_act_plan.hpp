// How the FP8 product with an epilogue runs: by few tokens, by tiles of one size,
// or split over the inner dimension (linear_act.hip).  Host code only.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace falq {
namespace {

// Which tile: the one whose rounds of the 256 CUs take least, by this model of
// them (us; gelu and z, 512 to 10240 columns, 4096 to 13824 K-bytes: within a
// tenth of the measured times, mostly).  A larger tile moves fewer bytes per
// product but leaves more of its last round empty, and where a CU holds one
// workgroup, all of a round's outputs are stored at once, with the matrix cores
// idle; where it holds two, one stores under the other's products.
//   8192 x 11008 x 4096 with gelu and z: 305 in 256 x 128, 342 in 256 x 256,
//     375 in 256 x 320 (a fifth round of 96 tiles), 345 in 128 x 128
//   4096 x 5120 x 13824: 187 in 256 x 320 (one round), 265 in 256 x 256
//   4096 x 4096 x 8192: 98 in 256 x 256 (one round), 110 in 256 x 128
//   1024 x 5120 x 5120 with gelu and z: 31.8 in 192 x 128, 36.2 in 256 x 128
//   512 x 11008 x 4096: 31.5 in 128 x 192, 36 in 256 x 128, 40 in 128 x 128
//   512 x 4096 x 4096: 15.5 in 64 x 64, 128 x 4096 x 4096: 10.0 in 32 x 64
// Fitted to 128 to 1024 tiles at 1024 and 4096 K-bytes, and 1056 and 4128 for rows
// that begin inside a 128-byte line (each step's chunk of a row then lies in two),
// between the times of a plain output and of gelu and z.
struct TileCost {
  int bm, bn;
  int per_cu;          // workgroups of a round on a CU
  float start, round;  // a launch, and a round of it, besides the K steps
  // a K step, at most one workgroup on a CU and at per_cu: rows of whole lines
  // and others
  struct {
    float alone, full;
  } step[2];
};
// Down to 128 x 128 linear_act_pipe, but for w8 and the small ones, which are
// linear_act_tile: more waves, which begin and end a tile faster.
enum TileKind {
  k256x320, k256, k256x128, k128x256, k192x128, k128x192w8, k128, k128w8, k64, k32x64, kTileKinds
};
constexpr TileCost kTile[kTileKinds] = {
    {256, 320, 1, 4.0f, 23.0f, {{1.47f, 1.47f}, {1.75f, 1.75f}}},
    {256, 256, 1, 3.0f, 15.0f, {{1.23f, 1.23f}, {1.50f, 1.50f}}},
    {256, 128, 2, 2.0f, 10.0f, {{0.70f, 1.42f}, {1.07f, 2.00f}}},
    {128, 256, 2, 2.0f, 10.0f, {{0.72f, 1.42f}, {1.08f, 2.00f}}},
    {192, 128, 2, 4.0f, 7.0f, {{0.52f, 1.08f}, {0.88f, 1.65f}}},
    {128, 192, 1, 2.5f, 6.0f, {{0.68f, 0.68f}, {0.85f, 0.85f}}},
    {128, 128, 2, 4.5f, 4.5f, {{0.39f, 0.78f}, {0.69f, 1.30f}}},
    {128, 128, 1, 3.0f, 3.0f, {{0.50f, 0.50f}, {0.68f, 0.68f}}},
    {64, 64, 2, 2.0f, 1.5f, {{0.27f, 0.50f}, {0.31f, 0.61f}}},
    {32, 64, 2, 2.0f, 1.0f, {{0.23f, 0.45f}, {0.23f, 0.48f}}}};
constexpr int kCUs = 256;
// the tiles of linear_act_pipe reach this far into a row by 32-bit offsets
constexpr int64_t kFarK = (int64_t)1 << 23;

int64_t tiles_of(TileKind k, int64_t M, int64_t N) {
  return ((M + kTile[k].bm - 1) / kTile[k].bm) * ((N + kTile[k].bn - 1) / kTile[k].bn);
}

float tile_cost(TileKind k, int64_t M, int64_t N, int64_t K) {
  const TileCost& t = kTile[k];
  const int64_t nt = tiles_of(k, M, N), cap = (int64_t)t.per_cu * kCUs, rest = nt % cap;
  // a grid holds fewer than 2^32 threads: very long outputs take large tiles
  if (k != k256 && nt >= 1 << 23) return HUGE_VALF;
  const auto& step = t.step[K % 128 != 0];
  const float last = rest == 0 ? 0.0f : rest <= kCUs ? step.alone : step.full;
  return t.start + (float)((nt + cap - 1) / cap) * t.round +
         (float)((K + 127) / 128) * ((float)(nt / cap) * step.full + last);
}

// How a product runs: by few tokens, by tiles of one kind, or by 128 x 128 tiles
// split over K (`split` parts, kc steps each).
struct Plan {
  int few = 0;
  TileKind kind = k256;
  int split = 1, kc = 0;
};

// waves of a workgroup of the few-token forms, which takes 16 columns
constexpr int kFewWaves[] = {0, 16, 8};

Plan plan_of(int64_t M, int64_t N, int64_t K) {
  Plan p;
  const int64_t steps = (K + 127) / 128;
  // few tokens: 4096 x 4096 5.6 us at 1 token and 6.6 at 16 (tiles of 32 x 64:
  // 9.5); at 32 tokens 7.7 against 9.6 while one workgroup per CU holds all
  // columns, 18.7 against 9.7 at 11008 columns
  // (a grid holds fewer than 2^32 threads: beyond that the tiles, which then are
  // too many for a split)
  if (K > 0 && M <= 16 && (N + 15) / 16 * kFewWaves[1] * 64 < (int64_t)1 << 32) p.few = 1;
  if (K > 0 && M > 16 && M <= 32 && N <= 16 * kCUs) p.few = 2;
  if (p.few) return p;
  float cost = HUGE_VALF;
  for (int k = 0; k < kTileKinds; ++k) {
    if (K > kFarK && k != k64 && k != k32x64) continue;
    const float c = tile_cost((TileKind)k, M, N, K);
    if (c >= cost) continue;
    cost = c;
    p.kind = (TileKind)k;
  }
  // few tiles and a long K: as many splits as give a workgroup to each CU, at
  // least 8 steps each, and the planes written and read once at 4 TB/s; two
  // launches, 8 us.  64 x
  // 5120 x 13824: 22.5 us in 6 splits, 32.5 whole; 100 x 4096 x 11008: 19.8 in
  // 8, 25.8 whole; 512 x 4096 x 4096 21.1 in 2, 15.5 whole.
  const int64_t nt = tiles_of(k128w8, M, N);
  const int64_t s = nt > 0 ? std::min<int64_t>(kCUs / nt, steps / 8) : 0;
  if (s >= 2) {
    const int64_t kc = (steps + s - 1) / s, parts = (steps + kc - 1) / kc;
    const float split = 8.0f + kTile[k128w8].step[0].alone * (float)kc +
                        (float)(parts * M * N) * 8.0f / 4e6f;
    if (parts >= 2 && split < cost) {
      p.split = (int)parts;
      p.kc = (int)kc;
    }
  }
  return p;
}

}  // namespace
}  // namespace falq
