// Layer norm over the last axis, forward and backward.
//
//   mu = sum x / d,  var = sum (x - mu)^2 / d,  rstd = 1 / sqrt(var + eps)
//   y  = (x - mu) rstd w + b
// and, with xh = (x - mu) rstd and g = dy w,
//   dx = rstd (g - sum(g) / d - xh sum(g xh) / d)
//   dw = sum over rows of dy xh,   db = sum over rows of dy.
// All sums are float32; the order of every sum is fixed by the shape.
#include "elem.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace falq {
namespace {

// sum of v over the workgroup (NT threads), in every thread
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum_f32(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += red[i];
    __syncthreads();
  }
  return v;
}

// One workgroup per row, which it reads three times.
template <class XT, class YT, int E>
__global__ __launch_bounds__(1024) void ln_fwd_long(const XT* __restrict__ x,
                                                    const float* __restrict__ w,
                                                    const float* __restrict__ b,
                                                    YT* __restrict__ y, float* __restrict__ mean,
                                                    float* __restrict__ rstd, int64_t T,
                                                    int64_t d, float eps) {
  __shared__ float red[16];
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x) {
    const XT* xr = x + row * d;
    YT* yr = y + row * d;
    float s = 0.0f;
    for (int64_t i = (int64_t)threadIdx.x * E; i < d; i += 1024 * E) {
      float v[E];
      load_elems<E>(xr + i, v);
#pragma unroll
      for (int e = 0; e < E; ++e) s += v[e];
    }
    const float mu = block_sum<1024>(s, red) / (float)d;
    s = 0.0f;
    for (int64_t i = (int64_t)threadIdx.x * E; i < d; i += 1024 * E) {
      float v[E];
      load_elems<E>(xr + i, v);
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(v[e] - mu, v[e] - mu, s);
    }
    const float rs = 1.0f / sqrtf(block_sum<1024>(s, red) / (float)d + eps);
    for (int64_t i = (int64_t)threadIdx.x * E; i < d; i += 1024 * E) {
      float v[E], t[E];
      load_elems<E>(xr + i, v);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = (v[e] - mu) * rs;
      if (w) {
        load_elems<E>(w + i, t);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= t[e];
      }
      if (b) {
        load_elems<E>(b + i, t);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] += t[e];
      }
      store_elems<E>(yr + i, v);
    }
    if (threadIdx.x == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
  }
}

// dx of one row per workgroup, which it reads twice
template <class XT, class GT, int E>
__global__ __launch_bounds__(1024) void ln_bwd_dx_long(
    const GT* dy, const XT* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ mean, const float* __restrict__ rstd, GT* dx, int64_t T,
    int64_t d) {
  __shared__ float red[16];
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x) {
    const float mu = mean[row], rs = rstd[row];
    const GT* gr = dy + row * d;
    const XT* xr = x + row * d;
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t i = (int64_t)threadIdx.x * E; i < d; i += 1024 * E) {
      float g[E], v[E], t[E];
      load_elems<E>(gr + i, g);
      load_elems<E>(xr + i, v);
      if (w) load_elems<E>(w + i, t);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (w) g[e] *= t[e];
        s1 += g[e];
        s2 = fmaf(g[e], (v[e] - mu) * rs, s2);
      }
    }
    const float c1 = block_sum<1024>(s1, red) / (float)d;
    const float c2 = block_sum<1024>(s2, red) / (float)d;
    for (int64_t i = (int64_t)threadIdx.x * E; i < d; i += 1024 * E) {
      float g[E], v[E], t[E];
      load_elems<E>(gr + i, g);
      load_elems<E>(xr + i, v);
      if (w) load_elems<E>(w + i, t);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (w) g[e] *= t[e];
        g[e] = rs * (g[e] - c1 - (v[e] - mu) * rs * c2);
      }
      store_elems<E>(dx + row * d + i, g);
    }
  }
}

// Columns of dw and db: a workgroup takes kColW columns and the rows of one
// strip, and writes its sums to row `strip` of the partials ([2 d] floats:
// dw, then db).
constexpr int kColRows = 8, kColLanes = 32;
template <class XT, class GT, int E>
__global__ __launch_bounds__(256) void ln_bwd_cols(
    const GT* __restrict__ dy, const XT* __restrict__ x, const float* __restrict__ mean,
    const float* __restrict__ rstd, float* __restrict__ part, int64_t T, int64_t d,
    int64_t rows_per_strip) {
  __shared__ float sw[kColRows][kColLanes * E], sb[kColRows][kColLanes * E];
  const int cl = threadIdx.x % kColLanes, rl = threadIdx.x / kColLanes;
  const int64_t col = ((int64_t)blockIdx.x * kColLanes + cl) * E;
  const int64_t r0 = blockIdx.y * rows_per_strip, r1 = min(T, r0 + rows_per_strip);
  float aw[E], ab[E];
#pragma unroll
  for (int e = 0; e < E; ++e) aw[e] = ab[e] = 0.0f;
  if (col < d)
    for (int64_t r = r0 + rl; r < r1; r += kColRows) {
      float g[E], v[E];
      load_elems<E>(dy + r * d + col, g);
      load_elems<E>(x + r * d + col, v);
      const float mu = mean[r], rs = rstd[r];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        aw[e] = fmaf(g[e], (v[e] - mu) * rs, aw[e]);
        ab[e] += g[e];
      }
    }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    sw[rl][cl * E + e] = aw[e];
    sb[rl][cl * E + e] = ab[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kColLanes * E; i += 256) {
    const int64_t c = (int64_t)blockIdx.x * kColLanes * E + i;
    if (c >= d) continue;
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int r = 0; r < kColRows; ++r) {
      a += sw[r][i];
      b += sb[r][i];
    }
    part[(int64_t)blockIdx.y * 2 * d + c] = a;
    part[(int64_t)blockIdx.y * 2 * d + d + c] = b;
  }
}

// workgroups of a row kernel: the work items of a launch fit 32 bits
unsigned row_grid(int64_t T) { return (unsigned)std::min<int64_t>(T, 1 << 20); }

struct Strips {
  int64_t n, rows;
};
Strips strips_of(int64_t T, int64_t d) {
  const int64_t cols = (d + 255) / 256;
  int64_t n = std::min<int64_t>((T + 31) / 32, std::max<int64_t>(1, 2048 / cols));
  n = std::max<int64_t>(1, std::min<int64_t>(n, 512));
  const int64_t rows = (T + n - 1) / n;
  return {rows ? (T + rows - 1) / rows : 0, rows};
}

template <class XT, class GT, int E>
hipError_t bwd(const GT* dy, const XT* x, const float* w, const float* mean, const float* rstd,
               int64_t T, int64_t d, GT* dx, float* dw, float* db, float* part, hipStream_t s) {
  if (dw || db) {
    const Strips st = strips_of(T, d);
    const dim3 grid((unsigned)((d + kColLanes * E - 1) / (kColLanes * E)), (unsigned)st.n);
    ln_bwd_cols<XT, GT, E><<<grid, 256, 0, s>>>(dy, x, mean, rstd, part, T, d, st.rows);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = launch_column_sum(part, st.n, d, 2, dw, db, s);
    if (e != hipSuccess) return e;
  }
  if (dx) ln_bwd_dx_long<XT, GT, E><<<row_grid(T), 1024, 0, s>>>(dy, x, w, mean, rstd, dx, T,
                                                              d);
  return hipGetLastError();
}

template <class XT, class GT>
hipError_t bwd_by_width(const void* dy, const void* x, const float* w, const float* mean,
                        const float* rstd, int64_t T, int64_t d, void* dx, float* dw, float* db,
                        float* part, hipStream_t s) {
  const GT* g = (const GT*)dy;
  const XT* v = (const XT*)x;
  return d % 8 == 0 ? bwd<XT, GT, 8>(g, v, w, mean, rstd, T, d, (GT*)dx, dw, db, part, s)
                    : bwd<XT, GT, 1>(g, v, w, mean, rstd, T, d, (GT*)dx, dw, db, part, s);
}

template <class XT, class YT>
hipError_t fwd(const void* x, const float* w, const float* b, int64_t T, int64_t d, float eps,
               void* y, float* mean, float* rstd, hipStream_t s) {
  if (d % 8 == 0)
    ln_fwd_long<XT, YT, 8><<<row_grid(T), 1024, 0, s>>>((const XT*)x, w, b, (YT*)y, mean, rstd, T,
                                                     d, eps);
  else
    ln_fwd_long<XT, YT, 1><<<row_grid(T), 1024, 0, s>>>((const XT*)x, w, b, (YT*)y, mean, rstd, T,
                                                     d, eps);
  return hipGetLastError();
}

// out[c] = sum over the P rows of part (row: nout * d floats), in a fixed order
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part,
                                                          int64_t P, int64_t d, int nout,
                                                          float* __restrict__ out0,
                                                          float* __restrict__ out1) {
  __shared__ float red[16][64];
  const int cl = threadIdx.x & 63, rl = threadIdx.x >> 6;
  const int64_t W = d * nout, c = (int64_t)blockIdx.x * 64 + cl;
  float a = 0.0f;
  if (c < W)
    for (int64_t p = rl; p < P; p += 16) a += part[p * W + c];
  red[rl][cl] = a;
  __syncthreads();
  if (rl == 0 && c < W) {
#pragma unroll
    for (int r = 1; r < 16; ++r) a += red[r][cl];
    float* o = c < d ? out0 : out1;
    if (o) o[c < d ? c : c - d] = a;
  }
}

}  // namespace

hipError_t launch_column_sum(const float* part, int64_t P, int64_t d, int nout, float* out0,
                             float* out1, hipStream_t s) {
  if (d == 0) return hipSuccess;
  column_sum_kernel<<<(unsigned)((d * nout + 63) / 64), 1024, 0, s>>>(part, P, d, nout, out0,
                                                                     out1);
  return hipGetLastError();
}

size_t layer_norm_bwd_ws_bytes(int64_t T, int64_t d) {
  return (size_t)strips_of(T, d).n * 2 * (size_t)d * 4;
}

hipError_t launch_layer_norm_fwd(const void* x, int xt, const float* w, const float* b, int64_t T,
                                 int64_t d, float eps, void* y, int yt, float* mean, float* rstd,
                                 hipStream_t s) {
  if (T == 0) return hipSuccess;
  if (xt == 0)
    return yt == 0 ? fwd<float, float>(x, w, b, T, d, eps, y, mean, rstd, s)
                   : fwd<float, __bf16>(x, w, b, T, d, eps, y, mean, rstd, s);
  return yt == 0 ? fwd<__bf16, float>(x, w, b, T, d, eps, y, mean, rstd, s)
                 : fwd<__bf16, __bf16>(x, w, b, T, d, eps, y, mean, rstd, s);
}

hipError_t launch_layer_norm_bwd(const void* dy, int gt, const void* x, int xt, const float* w,
                                 const float* mean, const float* rstd, int64_t T, int64_t d,
                                 void* dx, float* dw, float* db, void* ws, hipStream_t s) {
  if (T == 0) {
    hipError_t e = dw ? launch_fill_f32(dw, d, 0.0f, s) : hipSuccess;
    if (e != hipSuccess) return e;
    return db ? launch_fill_f32(db, d, 0.0f, s) : hipSuccess;
  }
  float* part = (float*)ws;
  if (xt == 0)
    return gt == 0
               ? bwd_by_width<float, float>(dy, x, w, mean, rstd, T, d, dx, dw, db, part, s)
               : bwd_by_width<float, __bf16>(dy, x, w, mean, rstd, T, d, dx, dw, db, part, s);
  return gt == 0 ? bwd_by_width<__bf16, float>(dy, x, w, mean, rstd, T, d, dx, dw, db, part, s)
                 : bwd_by_width<__bf16, __bf16>(dy, x, w, mean, rstd, T, d, dx, dw, db, part, s);
}

}  // namespace falq
