// Backward of a linear layer's epilogue: with z = acc + bias, y = act(z) + residual,
//   dz = dy act'(z),   dbias = sum over rows of dz   (the residual's gradient is dy).
//
// A workgroup takes kLanes * E columns and one strip of rows: each lane keeps
// its columns' dbias in float32 registers over its rows, the row lanes join
// in LDS, and the strips in the fixed-order column sum.  Bound by memory: dy and
// z read, dz written once (8192 x 11008, gelu, fp32 dy, bf16 z: 175 us, 5.2 TB/s;
// 217 where a lane stores 32 bytes in two halves, 188 without the streaming hint).
#include "activation.hpp"
#include "elem.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace falq {
namespace {

constexpr int kLanes = 32;

// part: the strips' sums, one row of d floats each (dbias itself with one strip)
template <class GT, class ZT, int E, int ACT, int kRows, bool STREAM, bool ODD>
__global__ __launch_bounds__(kRows * kLanes) void act_bwd_kernel(
    const GT* dy, const ZT* __restrict__ z, GT* dz, float* __restrict__ part, int64_t T, int64_t d,
    int64_t rows_per_strip) {
  __shared__ float sb[kRows][kLanes * E];
  const int cl = threadIdx.x % kLanes, rl = threadIdx.x / kLanes;
  const Piece<E, ODD> p(((uint32_t)blockIdx.x * kLanes + cl) * E, (uint32_t)d);
  const int64_t r0 = blockIdx.y * rows_per_strip, r1 = min(T, r0 + rows_per_strip);
  float ab[E];
#pragma unroll
  for (int e = 0; e < E; ++e) ab[e] = 0.0f;
  if (p.any) {
#pragma unroll 2
    for (int64_t r = r0 + rl; r < r1; r += kRows) {
      Raw<GT, E> gr;
      Raw<ZT, E> v;
      gr.template load<STREAM>(dy + r * d + p.base);
      if constexpr (ACT != kNone) v.template load<STREAM>(z + r * d + p.base);
      float g[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        g[e] = gr[e];
        if constexpr (ACT != kNone) g[e] *= act_slope<ACT, GT>(v[e]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) ab[e] += g[e];
      if (dz) p.template store<STREAM>(dz + r * d, g);
    }
  }
  if (!part) return;
#pragma unroll
  for (int e = 0; e < E; ++e)                  // elements before the piece's own: none's
    if (p.own(e)) sb[rl][cl * E + e - p.over] = ab[e];
  __syncthreads();
  for (int i = threadIdx.x; i < kLanes * E; i += kRows * kLanes) {
    const int64_t c = (int64_t)blockIdx.x * kLanes * E + i;
    if (c >= d) continue;
    float b = 0.0f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) b += sb[r][i];
    part[(int64_t)blockIdx.y * d + c] = b;
  }
}

struct Strips {
  int64_t n, rows;
};
// Up to kShort rows one strip of 32 row lanes writes dbias itself: no second
// launch and no workspace.
constexpr int kShort = 256;
Strips strips_of(int64_t T, int64_t d) {
  if (T <= kShort) return {1, T};
  const int64_t per = kLanes * 4;
  const int64_t cols = std::max<int64_t>(1, (d + per - 1) / per);
  const int64_t n = std::min<int64_t>({(T + 15) / 16, (4096 + cols - 1) / cols, 1024});
  const int64_t rows = (T + n - 1) / n;
  return {(T + rows - 1) / rows, rows};
}

template <class GT, class ZT, int E, int kRows, bool STREAM, bool ODD>
hipError_t by_act(const GT* dy, const ZT* z, int act, int64_t T, int64_t d, GT* dz, float* part,
                  hipStream_t s) {
  const Strips st = strips_of(T, d);
  const dim3 grid((unsigned)((d + kLanes * E - 1) / (kLanes * E)), (unsigned)st.n);
#define FALQ_ACT(A)                                                                         \
  case A:                                                                                   \
    act_bwd_kernel<GT, ZT, E, A, kRows, STREAM, ODD>                                        \
        <<<grid, kRows * kLanes, 0, s>>>(dy, z, dz, part, T, d, st.rows);                   \
    break;
  switch (act) {
    FALQ_ACT(kNone) FALQ_ACT(kRelu) FALQ_ACT(kGelu) FALQ_ACT(kGeluTanh) FALQ_ACT(kSilu)
    default: return hipErrorInvalidValue;
  }
#undef FALQ_ACT
  return hipGetLastError();
}

template <class GT, class ZT, int E, bool ODD>
hipError_t by_rows(const GT* dy, const ZT* z, int act, int64_t T, int64_t d, GT* dz, float* part,
                   hipStream_t s) {
  if (T <= kShort) return by_act<GT, ZT, E, 32, false, ODD>(dy, z, act, T, d, dz, part, s);
  // the streaming hint needs whole lines
  if constexpr (!ODD)
    if (T * d * (int64_t)(2 * sizeof(GT) + sizeof(ZT)) > kStreamBytes)
      return by_act<GT, ZT, E, 8, true, false>(dy, z, act, T, d, dz, part, s);
  return by_act<GT, ZT, E, 8, false, ODD>(dy, z, act, T, d, dz, part, s);
}

template <class GT, class ZT>
hipError_t by_width(const void* dy, const void* z, int act, int64_t T, int64_t d, void* dz,
                    float* part, hipStream_t s) {
  constexpr int E = sizeof(GT) + sizeof(ZT) == 4 ? 8 : 4;
  const GT* g = (const GT*)dy;
  const ZT* v = (const ZT*)z;
  if (d % 8 == 0) return by_rows<GT, ZT, E, false>(g, v, act, T, d, (GT*)dz, part, s);
  return d >= 4 ? by_rows<GT, ZT, 4, true>(g, v, act, T, d, (GT*)dz, part, s)
                : by_rows<GT, ZT, 1, true>(g, v, act, T, d, (GT*)dz, part, s);
}

}  // namespace

size_t linear_act_bwd_ws_bytes(int64_t T, int64_t d) {
  const int64_t n = strips_of(T, d).n;
  return n == 1 ? 0 : (size_t)n * (size_t)d * 4;
}

hipError_t launch_linear_act_bwd(const void* dy, int gt, const void* z, int zt, int64_t T,
                                 int64_t d, int act, void* dz, float* dbias, void* ws,
                                 hipStream_t s) {
  if (d == 0) return hipSuccess;
  if (T == 0) return dbias ? launch_fill_f32(dbias, d, 0.0f, s) : hipSuccess;
  const int64_t n = strips_of(T, d).n;
  float* part = n > 1 && dbias ? (float*)ws : dbias;
  hipError_t e;
  if (gt == 0)
    e = zt == 0 ? by_width<float, float>(dy, z, act, T, d, dz, part, s)
                : by_width<float, __bf16>(dy, z, act, T, d, dz, part, s);
  else
    e = zt == 0 ? by_width<__bf16, float>(dy, z, act, T, d, dz, part, s)
                : by_width<__bf16, __bf16>(dy, z, act, T, d, dz, part, s);
  if (e != hipSuccess || !dbias || n == 1) return e;
  return launch_column_sum(part, n, d, 1, dbias, nullptr, s);
}

}  // namespace falq
