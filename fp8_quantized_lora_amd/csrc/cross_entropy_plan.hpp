// How the cross entropy over the vocabulary and its gradient run (cross_entropy.hip).
// Host code only.
#pragma once

#include "linear_act_plan.hpp"

#include <cstddef>

namespace falq {
namespace {

// The forward's tiles, by the model of linear_act_plan.hpp with its own costs: the
// products as float16 take twice the steps' time, and there is nothing to store.
//   4096 x 32000 x 4096: 747 us in 256 x 256, 827 in 128 x 128
//   4096 x 50000 x 1024: 386 and 365; 333 x 131071 x 1040 174 and 109
//   128 x 32000 x 4096: 35 in 128 x 128, 50 in 64 x 64; 64 tokens 34 and 26
//   17 x 32000 x 4096: 26 in 64 x 64, 23 in 32 x 64; 1 token 21.3 (with the weight
//   streamed through the registers as in linear_act_few.hpp 23.6, and 31 for 16)
enum LossKind { kLoss256, kLoss128, kLoss64, kLoss32x64, kLossKinds };
constexpr TileCost kLossTile[kLossKinds] = {
    {256, 256, 1, 5.0f, 8.0f, {{2.65f, 2.65f}, {2.90f, 2.90f}}},
    {128, 128, 2, 5.0f, 2.3f, {{0.82f, 1.58f}, {0.90f, 1.70f}}},
    {64, 64, 2, 4.0f, 1.2f, {{0.35f, 0.62f}, {0.38f, 0.68f}}},
    {32, 64, 2, 6.0f, 0.8f, {{0.25f, 0.39f}, {0.28f, 0.43f}}}};
LossKind loss_kind(int64_t T, int64_t V, int64_t d) {
  LossKind best = kLoss64;
  float cost = HUGE_VALF;
  for (int k = 0; k < kLossKinds; ++k) {
    const TileCost& t = kLossTile[k];
    const int64_t nt = ((T + t.bm - 1) / t.bm) * ((V + t.bn - 1) / t.bn);
    const float c = cost_of(t, nt, d);
    if (nt >= 1 << 23 || c >= cost) continue;
    cost = c;
    best = (LossKind)k;
  }
  return best;
}

// G's tiles for gradients in bfloat16 (in float32 they are the forward's), by
// linear_act_plan.hpp's costs, those kinds that are cheapest somewhere:
//   4096 x 32000 x 4096: 431 us in 256 x 256, 469 in 192 x 128, 466 in 256 x 128, 559 in
//     128 x 128; 512 tokens 60, 61, 57 and 62
//   4096 x 50000 x 1024: 258 in 192 x 128, 294 in 256 x 128, 321 in 256 x 256; 333 x 131071
//     x 1040 76, 94 and 113 (128 x 128: 97)
//   128 x 16000 x 4096: 17 in 64 x 64, 20 in 128 x 128; 17 tokens 12.1 in 32 x 64, 12.8
enum GradKind {
  kGrad256, kGrad256x128, kGrad192x128, kGrad128, kGrad64, kGrad32x64, kGradKinds
};
constexpr TileKind kGradTile[kGradKinds] = {k256, k256x128, k192x128, k128, k64, k32x64};
GradKind grad_kind(int64_t T, int64_t n, int64_t d) {
  GradKind best = kGrad64;
  float cost = HUGE_VALF;
  for (int k = 0; k < kGradKinds; ++k) {
    const float c = tile_cost(kGradTile[k], T, n, d);
    if (c >= cost) continue;
    cost = c;
    best = (GradKind)k;
  }
  return best;
}

int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up(int64_t a, int64_t b) { return ceil_div64(a, b) * b; }

// Rows are taken in strips, so that no workspace grows with T beyond a strip's.  (With V the
// forward's does: 8 bytes for a row's 64 to 256 columns, 67 MB of 16384 x 131072.)
constexpr int64_t kStrip = 16384;
int64_t strip_of(int64_t T) { return std::min(T, kStrip); }

// runs of columns of the forward's partial sums: the tiles'
int64_t runs_of(int64_t T, int64_t d, int64_t V) {
  return ceil_div64(V, kLossTile[loss_kind(T, V, d)].bn);
}

// pieces of the vocabulary: as many as keep G (and, for float32 gradients, what its rounding
// leaves) within kPiece bytes, of one width, a multiple of 64.  Larger ones than the
// last-level cache holds cost G's way to memory and back, smaller ones more launches' ends
// and dx's sums read and written again: 4096 x 4096 x 32000 1276 us with 512 MB, 1279 with
// 256, 1323 with 128, 1374 with 64; 8192 tokens 2522, 2593, 2756 and 2948; 4096 x 1024 x
// 50000 716, 743, 766 and 800.
constexpr int64_t kPiece = (int64_t)512 << 20;
// bytes: of an element of G
int64_t piece_width(int64_t T, int64_t V, int bytes) {
  const int64_t most = std::clamp<int64_t>(kPiece / (bytes * T), 2048, 1 << 21);
  return up(ceil_div64(V, ceil_div64(V, most)), 64);
}

// dx's tiles and splits over the piece's columns, by the same model; a split's sums are
// written and read once at 4 TB/s and joined by a launch of their own.
//   32000 columns: 4096 x 4096 800 us in 256 x 256 (256 x 128: 830); 2048 x 4096 420 in
//     256 x 128 (588; 128 x 128: 483)
//   1024 x 4096: 222 in 2 splits of 256 x 128, 252 in 128 x 128 whole; 2048 x 1024 120
//     in 4, 205 whole
//   128 x 4096: 45 in 8 splits of 128 x 128, 67 of 64 x 64; 64 x 4096: 39 and 37; 17 x
//     4096: 36 in 8 of 64 x 64, 29 of 32 x 64
//   131071 columns, 333 x 1040: 127 in 8 splits of 128 x 128, 161 of 256 x 128
enum DxKind { kDx256, kDx256x128, kDx128, kDx64, kDx32x64, kDxKinds };
constexpr TileCost kDxTile[kDxKinds] = {
    {256, 256, 1, 3.0f, 15.0f, {{1.50f, 1.50f}, {1.50f, 1.50f}}},
    {256, 128, 2, 2.0f, 10.0f, {{0.80f, 1.60f}, {0.80f, 1.60f}}},
    {128, 128, 2, 4.5f, 4.5f, {{0.47f, 0.94f}, {0.47f, 0.94f}}},
    {64, 64, 2, 2.0f, 1.5f, {{0.32f, 0.42f}, {0.32f, 0.42f}}},
    {32, 64, 2, 2.0f, 1.0f, {{0.27f, 0.35f}, {0.27f, 0.35f}}}};

struct BwdPlan {
  int64_t width;
  DxKind kind;
  int splits, kc;                                            // kc K steps each
  size_t g, sums, part, rows;                           // bytes, multiples of 256
  size_t bytes() const { return g + sums + part + rows; }
};
BwdPlan bwd_plan(int64_t T, int64_t d, int64_t V, int dx_type) {
  BwdPlan p;
  // (float32 gradients: of G and of what its rounding leaves)
  const int bytes = dx_type == 0 ? 4 : 2;
  p.width = piece_width(T, V, bytes);
  p.kind = kDx64;
  p.splits = 1;
  p.kc = 0;
  const int64_t steps = ceil_div64(p.width, 64);
  float cost = HUGE_VALF;
  for (int k = 0; k < kDxKinds; ++k) {
    const TileCost& t = kDxTile[k];
    const int64_t nt = ceil_div64(T, t.bm) * ceil_div64(d, t.bn);
    // (pipelined tiles reach this far into a row of G by 32-bit offsets)
    if (p.width * 2 > kFarK && k < kDx64) continue;
    for (int s = 1; s <= 32; s *= 2) {
      if (s > 1 && (k == kDx256 || steps / s < 8)) break;
      const int64_t kc = ceil_div64(steps, s);
      const float join = s == 1 ? 0.0f : 3.0f + (float)(s * T * d) * 8.0f / 4e6f;
      const float c = cost_of(t, nt * s, kc * 128) + join;
      if (nt * s >= 1 << 22 || c >= cost) continue;
      cost = c;
      p.kind = (DxKind)k;
      p.splits = s;
      p.kc = (int)kc;
    }
  }
  p.g = (size_t)up(T * p.width * bytes, 256);
  // float32 gradients collect in place
  p.sums = dx_type != 0 && p.width < V ? (size_t)up(T * d * 4, 256) : 0;
  p.part = p.splits > 1 ? (size_t)up(p.splits * T * d * 4, 256) : 0;
  p.rows = (size_t)up(T * 16, 256);                          // a GradRow each
  return p;
}

}  // namespace
}  // namespace falq
