// How the product of FP4 operands runs, by the model of linear_act_plan.hpp with the
// costs of its own kernels (K in bytes, two elements each).  Host code only.
#pragma once

#include "linear_act_plan.hpp"

namespace falq {
namespace {

// Tiles of 256 x 128, two on a CU: one workgroup's epilogue runs under the other's
// products, which with FP4 take half the time for the same outputs: 8192 x 11008 x 4096
// with gelu and z 213 us, 257 in 256 x 256 alone on a CU; 189 and 207 without; 8192^3 250
// and 240.  128 x 128, which load more for a product, where 256 x 128 leave CUs empty:
// 4096 x 5120 x 13824 141 and 149, 1024 x 11008 x 4096 with gelu and z 36 and 40, 1024
// x 4096 x 4096 13.7 and 20.9.  64 x 64 and 32 x 64 where those do: 512 x 4096 x 4096
// 11.5 (128 x 128: 12.0), 256 x 11008 x 4096 17.7 (12.9), 128 x 4096 x 4096 8.5 and 7.1
// (11.1), 37 x 11008 x 4064 8.6 and 8.6 (12.1).
enum MxKind { kMx256x128, kMx128, kMx64, kMx32x64, kMxKinds };
constexpr TileCost kMxTile[kMxKinds] = {
    {256, 128, 2, 7.0f, 8.0f, {{0.70f, 1.84f}, {0.91f, 2.30f}}},
    {128, 128, 2, 7.5f, 4.0f, {{0.34f, 0.98f}, {0.44f, 1.22f}}},
    {64, 64, 2, 2.5f, 2.8f, {{0.25f, 0.44f}, {0.31f, 0.55f}}},
    {32, 64, 2, 4.0f, 0.8f, {{0.20f, 0.30f}, {0.25f, 0.38f}}}};

struct MxPlan {
  int few = 0;
  MxKind kind = kMx256x128;
  int split = 1, kc = 0;
};

MxPlan mx_plan_of(int64_t M, int64_t N, int64_t K) {
  MxPlan p;
  const int64_t steps = (K + 127) / 128;
  const auto tiles = [&](int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  // few tokens as in plan_of: 16 x 4096 x 4096 4.4 us (32 x 64: 6.8), 32 tokens 5.4 (6.8)
  if (K > 0 && M <= 16 && (N + 15) / 16 * kFewWaves[1] * 64 < (int64_t)1 << 32) p.few = 1;
  if (K > 0 && M > 16 && M <= 32 && N <= 16 * kCUs) p.few = 2;
  if (p.few) return p;
  float cost = HUGE_VALF;
  for (int k = 0; k < kMxKinds; ++k) {
    const TileCost& t = kMxTile[k];
    const int64_t nt = tiles(t.bm, t.bn);
    if (K > kFarK && k < kMx64) continue;
    if (k != kMx256x128 && nt >= 1 << 23) continue;
    const float c = cost_of(t, nt, K);
    if (c >= cost) continue;
    cost = c;
    p.kind = (MxKind)k;
  }
  // few tiles and a long K: 128 x 128 tiles of eight waves split over it, as plan_of
  const int64_t nt = tiles(128, 128), s = nt > 0 ? std::min<int64_t>(kCUs / nt, steps / 8) : 0;
  if (s >= 2) {
    const int64_t kc = (steps + s - 1) / s, parts = (steps + kc - 1) / kc;
    const float split = 8.0f + 0.6f * (float)kc + (float)(parts * M * N) * 8.0f / 4e6f;
    if (parts >= 2 && split < cost) {
      p.split = (int)parts;
      p.kc = (int)kc;
    }
  }
  return p;
}

}  // namespace
}  // namespace falq
