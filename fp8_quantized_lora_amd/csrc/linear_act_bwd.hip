// Backward of a linear layer's epilogue: with z = acc + bias, y = act(z) + residual,
//   dz = dy act'(z),   dbias = sum over rows of dz   (the residual's gradient is dy).
//
// A workgroup takes kLanes * E columns and one strip of rows: each lane keeps
// its columns' dbias in float32 registers over its rows, the row lanes join
// in LDS, and the strips in the fixed-order column sum.
#include "activation.hpp"
#include "elem.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace falq {
namespace {

constexpr int kRows = 8, kLanes = 32;

template <class GT, class ZT, int E, int ACT>
__global__ __launch_bounds__(256) void act_bwd_kernel(const GT* dy, const ZT* __restrict__ z,
                                                      GT* dz, float* __restrict__ part, int64_t T,
                                                      int64_t d, int64_t rows_per_strip) {
  __shared__ float sb[kRows][kLanes * E];
  const int cl = threadIdx.x % kLanes, rl = threadIdx.x / kLanes;
  const int64_t col = ((int64_t)blockIdx.x * kLanes + cl) * E;
  const int64_t r0 = blockIdx.y * rows_per_strip, r1 = min(T, r0 + rows_per_strip);
  float ab[E];
#pragma unroll
  for (int e = 0; e < E; ++e) ab[e] = 0.0f;
  if (col < d) {
#pragma unroll 2
    for (int64_t r = r0 + rl; r < r1; r += kRows) {
      float g[E], v[E];
      load_elems<E>(dy + r * d + col, g);
      if constexpr (ACT != kNone) {
        load_elems<E>(z + r * d + col, v);
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] *= act_slope<ACT>(v[e]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) ab[e] += g[e];
      store_elems<E>(dz + r * d + col, g);
    }
  }
  if (!part) return;
#pragma unroll
  for (int e = 0; e < E; ++e) sb[rl][cl * E + e] = ab[e];
  __syncthreads();
  for (int i = threadIdx.x; i < kLanes * E; i += 256) {
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
Strips strips_of(int64_t T, int64_t d) {
  const int64_t per = d % 8 == 0 ? kLanes * 8 : kLanes;
  const int64_t cols = std::max<int64_t>(1, (d + per - 1) / per);
  int64_t n = std::min<int64_t>((T + 2 * kRows - 1) / (2 * kRows), (4096 + cols - 1) / cols);
  n = std::max<int64_t>(1, std::min<int64_t>(n, 1024));
  const int64_t rows = (T + n - 1) / n;
  return {rows ? (T + rows - 1) / rows : 0, rows};
}

template <class GT, class ZT, int E>
hipError_t by_act(const GT* dy, const ZT* z, int act, int64_t T, int64_t d, GT* dz, float* part,
                  hipStream_t s) {
  const Strips st = strips_of(T, d);
  const dim3 grid((unsigned)((d + kLanes * E - 1) / (kLanes * E)), (unsigned)st.n);
#define FALQ_ACT(A)                                                                      \
  case A:                                                                                \
    act_bwd_kernel<GT, ZT, E, A><<<grid, 256, 0, s>>>(dy, z, dz, part, T, d, st.rows);   \
    break;
  switch (act) {
    FALQ_ACT(kNone) FALQ_ACT(kRelu) FALQ_ACT(kGelu) FALQ_ACT(kGeluTanh) FALQ_ACT(kSilu)
    default: return hipErrorInvalidValue;
  }
#undef FALQ_ACT
  return hipGetLastError();
}

template <class GT, class ZT>
hipError_t by_width(const void* dy, const void* z, int act, int64_t T, int64_t d, void* dz,
                    float* part, hipStream_t s) {
  return d % 8 == 0 ? by_act<GT, ZT, 8>((const GT*)dy, (const ZT*)z, act, T, d, (GT*)dz, part, s)
                    : by_act<GT, ZT, 1>((const GT*)dy, (const ZT*)z, act, T, d, (GT*)dz, part, s);
}

}  // namespace

size_t linear_act_bwd_ws_bytes(int64_t T, int64_t d) {
  return (size_t)strips_of(T, d).n * (size_t)d * 4;
}

hipError_t launch_linear_act_bwd(const void* dy, int gt, const void* z, int zt, int64_t T,
                                 int64_t d, int act, void* dz, float* dbias, void* ws,
                                 hipStream_t s) {
  if (d == 0) return hipSuccess;
  if (T == 0) return dbias ? launch_fill_f32(dbias, d, 0.0f, s) : hipSuccess;
  float* part = dbias ? (float*)ws : nullptr;
  hipError_t e;
  if (gt == 0)
    e = zt == 0 ? by_width<float, float>(dy, z, act, T, d, dz, part, s)
                : by_width<float, __bf16>(dy, z, act, T, d, dz, part, s);
  else
    e = zt == 0 ? by_width<__bf16, float>(dy, z, act, T, d, dz, part, s)
                : by_width<__bf16, __bf16>(dy, z, act, T, d, dz, part, s);
  if (e != hipSuccess || !dbias) return e;
  return launch_column_sum(part, strips_of(T, d).n, d, 1, dbias, nullptr, s);
}

}  // namespace falq
