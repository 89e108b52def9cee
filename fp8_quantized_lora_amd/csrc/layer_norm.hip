// Layer norm over the last axis, forward and backward.
//
//   mu = sum x / d,  var = sum (x - mu)^2 / d,  rstd = 1 / sqrt(var + eps)
//   y  = (x - mu) rstd w + b
// and, with xh = (x - mu) rstd and g = dy w,
//   dx = rstd (g - sum(g) / d - xh sum(g xh) / d)
//   dw = sum over rows of dy xh,   db = sum over rows of dy.
// All sums are float32; the order of every sum is fixed by the shape and types.
//
// Both are bound by memory: x read and y written once (4096 x 5120, fp32 to
// bf16: 25.3 us, 5.0 TB/s); dy and x read and dx written once (8192 x 4096, fp32
// dy, bf16 x: 65.7 us, 5.1 TB/s; a copy on this card reaches 5.1 to 5.4; x as an 8-bit
// checkpoint 54 us on the GPU, 5.6 TB/s).  A row
// lies in the registers of a group of 64 to 1024 threads from its one read on;
// rows too long for that (32768 elements forward, 16384 backward) are read again
// for each pass.
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
    const GT* dy, const XT* __restrict__ x, const uint8_t* __restrict__ xs,
    const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
    GT* dx, int64_t T, int64_t d) {
  __shared__ float red[16];
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x) {
    const float mu = mean[row], rs = rstd[row];
    const GT* gr = dy + row * d;
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t i = (int64_t)threadIdx.x * E; i < d; i += 1024 * E) {
      float g[E], v[E], t[E];
      load_elems<E>(gr + i, g);
      load_row_elems<E>(x, xs, row, d, i, v);
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
      load_row_elems<E>(x, xs, row, d, i, v);
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

// A row per group of nt threads (a multiple of 64, G groups in the workgroup),
// in registers: thread t holds elements (c nt + t) E .. + E for c < C.
// Sums of the row over the group: within the waves, then over the group's
// waves in LDS; `red` alternates between two halves, so one barrier each.
struct Group {
  int nt, t, first, waves, wave;
  __device__ __forceinline__ explicit Group(int nt_)
      : nt(nt_), t((int)threadIdx.x % nt_), first((int)threadIdx.x / nt_ * (nt_ / 64)),
        waves(nt_ / 64), wave((int)threadIdx.x / 64) {}
  template <int E>
  __device__ __forceinline__ uint32_t at(int c) const {
    return ((uint32_t)c * (uint32_t)nt + (uint32_t)t) * E;
  }
  __device__ __forceinline__ int index() const { return (int)threadIdx.x / nt; }
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N], float (*red)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum_f32(v[i]);
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave][i] = v[i];
    __syncthreads();
    // one lane per wave of the group (at most 16): one read, four additions
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = row_sum_f32(lane < waves ? red[first + lane][i] : 0.0f);
  }
};

template <class XT, class YT, int E, int C, bool STREAM, bool ODD>
__global__ __launch_bounds__(1024) void ln_fwd_rows(const XT* __restrict__ x,
                                                    const float* __restrict__ w,
                                                    const float* __restrict__ b,
                                                    YT* __restrict__ y, float* __restrict__ mean,
                                                    float* __restrict__ rstd, int64_t T, int d,
                                                    float eps, int nt) {
  __shared__ float red[2][16][1];
  const Group gr(nt);
  const int G = (int)blockDim.x / nt;
  const float inv = 1.0f / (float)d;
  for (int64_t r0 = (int64_t)blockIdx.x * G; r0 < T; r0 += (int64_t)gridDim.x * G) {
    // the wave's row, in a scalar register: one base address for all chunks
    const int64_t row = __builtin_amdgcn_readfirstlane((int)(r0 + gr.index()));
    const bool live = row < T;
    const XT* xr = x + (live ? row : T - 1) * d;
    YT* yr = y + row * d;
    Raw<XT, E> raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<E, ODD> p(gr.at<E>(c), d);
      if (p.any) raw[c].template load<STREAM>(xr + p.base);
    }
    float v[C][E], s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<E, ODD> p(gr.at<E>(c), d);
      if (p.any)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v[c][e] = raw[c][e];
          if (p.own(e)) s[0] += v[c][e];
        }
    }
    gr.sum(s, red[0]);
    const float mu = s[0] * inv;
    s[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<E, ODD> p(gr.at<E>(c), d);
      if (p.any)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v[c][e] -= mu;
          if (p.own(e)) s[0] = fmaf(v[c][e], v[c][e], s[0]);
        }
    }
    gr.sum(s, red[1]);
    const float rs = 1.0f / sqrtf(s[0] * inv + eps);
    if (live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const Piece<E, ODD> p(gr.at<E>(c), d);
        if (!p.any) continue;
        float f[E];
        if (w) {
          load_elems<E>(w + p.base, f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[c][e] = v[c][e] * rs * f[e];
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) v[c][e] *= rs;
        }
        if (b) {
          load_elems<E>(b + p.base, f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[c][e] += f[e];
        }
        p.template store<STREAM>(yr, v[c]);
      }
      if (gr.t == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
      }
    }
  }
}

// dx, and the sums of dw and db over the workgroup's rows (to its row of the
// partials, [2 d] floats: dw, then db), in one pass: the next row's loads are
// sent before the current row's sums are waited for, and the current row stays
// in registers as it lies in memory.
template <class XT, class GT, int E, int C, int MOST, bool STREAM, bool ODD>
__global__ __launch_bounds__(MOST) void ln_bwd_rows(const GT* dy, const XT* __restrict__ x,
                                                    const uint8_t* __restrict__ xs,
                                                    const float* __restrict__ w,
                                                    const float* __restrict__ mean,
                                                    const float* __restrict__ rstd, GT* dx,
                                                    float* __restrict__ part, int64_t T, int d,
                                                    int nt) {
  // two fp32 rows of 16 elements a thread do not fit 128 registers together
  constexpr bool kAhead = !(C * E == 16 && MOST == 1024 && sizeof(XT) + sizeof(GT) == 8);
  __shared__ float red[2][16][2];
  extern __shared__ float join[];                            // C E nt (G / 2) floats
  const Group gr(nt);
  const int G = (int)blockDim.x / nt;
  const float inv = 1.0f / (float)d;
  float wv[C][E], aw[C][E], ab[C][E];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      wv[c][e] = 1.0f;
      aw[c][e] = ab[c][e] = 0.0f;
    }
    const Piece<E, ODD> p(gr.at<E>(c), d);
    if (w && p.any) load_elems<E>(w + p.base, wv[c]);
  }
  // a row, its statistics in scalar registers (a wave is within one row);
  // zeros in the threads past its end
  struct Row {
    Raw<GT, E> g[C];
    RowElems<XT, E, ODD> v[C];
    float mu, rs;
  };
  auto load = [&](Row& o, int64_t r) {
    const int64_t row = __builtin_amdgcn_readfirstlane((int)(r < T ? r : T - 1));
    const GT* dyr = dy + row * d;
    const auto xr = RowElems<XT, E, ODD>::at(x, xs, row, d);
    o.mu = mean[row];
    o.rs = rstd[row];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<E, ODD> p(gr.at<E>(c), d);
      if (p.any) {
        o.g[c].template load<STREAM>(dyr + p.base);
        o.v[c].template load<STREAM>(xr, p.base);
      } else {
        o.g[c].clear();
        o.v[c].clear();
      }
    }
  };
  const int64_t stride = (int64_t)gridDim.x * G;
  auto work = [&](const Row& o, Row& next, int64_t r0, int half) {
    const int64_t row = __builtin_amdgcn_readfirstlane((int)(r0 + gr.index()));
    const bool live = row < T;
    GT* dxr = dx + row * d;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<E, ODD> p(gr.at<E>(c), d);
      if (p.any)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (!p.own(e)) continue;
          const float g = o.g[c][e], xh = (o.v[c][e] - o.mu) * o.rs, gw = g * wv[c][e];
          s[0] += gw;
          s[1] = fmaf(gw, xh, s[1]);
          if (live) {
            aw[c][e] = fmaf(g, xh, aw[c][e]);
            ab[c][e] += g;
          }
        }
    }
    if (kAhead && r0 + stride < T) load(next, row + stride);
    gr.sum(s, red[half]);
    if (live && dx) {
      const float c1 = s[0] * inv, c2 = s[1] * inv;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const Piece<E, ODD> p(gr.at<E>(c), d);
        if (!p.any) continue;
        float out[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
          out[e] = o.rs * (o.g[c][e] * wv[c][e] - c1 - (o.v[c][e] - o.mu) * o.rs * c2);
        p.template store<STREAM>(dxr, out);
      }
    }
    if (!kAhead && r0 + stride < T) load(next, row + stride);
  };
  Row a, b;
  int64_t r0 = (int64_t)blockIdx.x * G;
  load(a, r0 + gr.index());
  while (r0 < T) {                                           // two rows a turn: no copies
    work(a, b, r0, 0);
    r0 += stride;
    if (r0 >= T) break;
    work(b, a, r0, 1);
    r0 += stride;
  }
  if (!part) return;
  // the groups' sums, upper half onto lower half until one is left
  for (int n = G; n > 1;) {
    const int keep = (n + 1) / 2;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float(&acc)[C][E] = k ? ab : aw;
      __syncthreads();
      if (gr.index() >= keep && gr.index() < n)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < E; ++e)
            join[(c * E + e) * (n - keep) * nt + (gr.index() - keep) * nt + gr.t] = acc[c][e];
      __syncthreads();
      if (gr.index() < n - keep)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < E; ++e)
            acc[c][e] += join[(c * E + e) * (n - keep) * nt + gr.index() * nt + gr.t];
    }
    n = keep;
  }
  if (gr.index() == 0) {
    float* to = part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<E, ODD> p(gr.at<E>(c), d);
      if (!p.any) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (!p.own(e)) continue;
        to[p.base + e] = aw[c][e];
        to[d + p.base + e] = ab[c][e];
      }
    }
  }
}

// Few rows (kShortRows): dx, dw and db in one launch and without a workspace.
// The first `row_blocks` workgroups form dx, a row per group; the others take
// 32 columns each and all rows, and write dw and db themselves: dw and db need
// only the forward's statistics, and the second read of dy and x comes from
// the caches.
constexpr int kShortCols = 32;
template <class XT, class GT, int E, int C, bool ODD>
__global__ __launch_bounds__(1024) void ln_bwd_short(
    const GT* dy, const XT* __restrict__ x, const uint8_t* __restrict__ xs,
    const float* __restrict__ w, const float* __restrict__ mean, const float* __restrict__ rstd,
    GT* dx, float* __restrict__ dw, float* __restrict__ db, int T, int d, int nt, int row_blocks) {
  if ((int)blockIdx.x < row_blocks) {
    __shared__ float red[16][2];
    const Group gr(nt);
    const int64_t at = (int64_t)blockIdx.x * ((int)blockDim.x / nt) + gr.index();
    const int64_t row = __builtin_amdgcn_readfirstlane((int)at);
    const bool live = row < T;
    const int64_t from = (live ? row : T - 1) * d;
    const float mu = mean[live ? row : T - 1], rs = rstd[live ? row : T - 1];
    float gw[C][E], xh[C][E], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<E, ODD> p(gr.at<E>(c), d);
      if (!p.any) continue;
      float f[E];
      load_elems<E>(dy + from + p.base, gw[c]);
      RowElems<XT, E, ODD> v;
      v.load(v.at(x, xs, live ? row : T - 1, d), p.base);
      if (w) load_elems<E>(w + p.base, f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (w) gw[c][e] *= f[e];
        xh[c][e] = (v[e] - mu) * rs;
        if (!p.own(e)) continue;
        s[0] += gw[c][e];
        s[1] = fmaf(gw[c][e], xh[c][e], s[1]);
      }
    }
    gr.sum(s, red);
    if (!live) return;
    const float inv = 1.0f / (float)d, c1 = s[0] * inv, c2 = s[1] * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Piece<E, ODD> p(gr.at<E>(c), d);
      if (!p.any) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) gw[c][e] = rs * (gw[c][e] - c1 - xh[c][e] * c2);
      p.store(dx + from, gw[c]);
    }
    return;
  }
  __shared__ float sums[2][32][kShortCols];
  const int cl = threadIdx.x % kShortCols, rl = threadIdx.x / kShortCols;
  const int lanes = (int)blockDim.x / kShortCols;            // at most 32
  const int col = ((int)blockIdx.x - row_blocks) * kShortCols + cl;
  float a = 0.0f, b = 0.0f;
  if (col < d) {
#pragma unroll 8
    for (int r = rl; r < T; r += lanes) {
      const float g = (float)dy[(int64_t)r * d + col];
      float v[1];
      load_row_elems<1>(x, xs, r, d, col, v);
      a = fmaf(g, (v[0] - mean[r]) * rstd[r], a);
      b += g;
    }
  }
  sums[0][rl][cl] = a;
  sums[1][rl][cl] = b;
  __syncthreads();
  if (rl < 2 && col < d) {
    float* o = rl ? db : dw;
    if (!o) return;
    float v = sums[rl][0][cl];
    for (int r = 1; r < lanes; ++r) v += sums[rl][r][cl];
    o[col] = v;
  }
}

// Columns of dw and db: a workgroup takes kColW columns and the rows of one
// strip, and writes its sums to row `strip` of the partials ([2 d] floats:
// dw, then db).
constexpr int kColRows = 8, kColLanes = 32;
template <class XT, class GT, int E>
__global__ __launch_bounds__(256) void ln_bwd_cols(
    const GT* __restrict__ dy, const XT* __restrict__ x, const uint8_t* __restrict__ xs,
    const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part,
    int64_t T, int64_t d, int64_t rows_per_strip) {
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
      load_row_elems<E>(x, xs, r, d, col, v);
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

// threads of a row that hold n elements each; 0: more than `most`
int row_threads(int64_t d, int n, int most) {
  const int64_t nt = (d + (int64_t)64 * n - 1) / ((int64_t)64 * n) * 64;
  return nt <= most ? (int)nt : 0;
}

// Workgroups of the backward, and rows of partials, at most: one per CU.  More
// hide no more latency (the next row is under way) and write more partials:
// 8192 x 4096 with bf16 x and fp32 dy 67.2 us with 256 workgroups of 512
// threads, 75.6 with 512, 83.1 with 1024; 78.3 with 128.
constexpr int kBwdBlocks = 256;

struct BwdPlan {
  int n, nt, G, blocks;                        // n elements a thread; 0: rows too long or short
};
// threads: of a workgroup of several rows.  512, or for an 8-bit checkpoint 1024, whose
// rows are fewer bytes under way, where there are rows for all: 8192 x 4096 with fp32 dy 62
// us (512: 67), with bf16 dy 41.8 (44.7), 2048 x 4096 20.4 (21.3).
BwdPlan bwd_plan(int64_t T, int64_t d, int threads = 512) {
  int n = 8, nt = row_threads(d, n, 1024);
  if (!nt) nt = row_threads(d, n = 16, 1024);
  if (!nt || d < 4) return {0, 0, 0, 0};
  if (T < (int64_t)kBwdBlocks * (threads / nt)) threads = 512;
  const int G = std::max(1, threads / nt);
  return {n, nt, G, (int)std::min<int64_t>((T + G - 1) / G, kBwdBlocks)};
}

template <class XT, class GT, int E, int C, bool STREAM, bool ODD>
hipError_t bwd_rows(const BwdPlan& p, const GT* dy, const XT* x, const uint8_t* xs, const float* w,
                    const float* mean, const float* rstd, int64_t T, int64_t d, GT* dx, float* part,
                    hipStream_t s) {
  const size_t lds = (size_t)C * E * (p.G / 2) * p.nt * 4;
  // a workgroup of at most 512 threads may use twice the registers
  if (p.nt * p.G <= 512)
    ln_bwd_rows<XT, GT, E, C, 512, STREAM, ODD><<<p.blocks, p.nt * p.G, lds, s>>>(
        dy, x, xs, w, mean, rstd, dx, part, T, (int)d, p.nt);
  else
    ln_bwd_rows<XT, GT, E, C, 1024, STREAM, ODD><<<p.blocks, p.nt * p.G, lds, s>>>(
        dy, x, xs, w, mean, rstd, dx, part, T, (int)d, p.nt);
  return hipGetLastError();
}

constexpr int64_t kShortRows = 1024;
bool bwd_short_fits(int64_t T, int64_t d) {
  return T <= kShortRows && d >= 4 && row_threads(d, 8, 1024) > 0;
}

template <class XT, class GT, int E, bool ODD>
hipError_t bwd_short(const GT* dy, const XT* x, const uint8_t* xs, const float* w,
                     const float* mean, const float* rstd, int64_t T, int64_t d, GT* dx, float* dw,
                     float* db, hipStream_t s) {
  const int nt = row_threads(d, 8, 1024), G = 1024 / nt;
  const int rows = dx ? (int)((T + G - 1) / G) : 0;
  const int cols = dw || db ? (int)((d + kShortCols - 1) / kShortCols) : 0;
  auto launch = [&](int row_blocks, int col_blocks) {
    if (row_blocks + col_blocks > 0)
      ln_bwd_short<XT, GT, E, 8 / E, ODD><<<row_blocks + col_blocks, nt * G, 0, s>>>(
          dy, x, xs, w, mean, rstd, dx, dw, db, (int)T, (int)d, nt, row_blocks);
  };
  if ((const GT*)dx == dy) {                   // in place: the columns are read first
    launch(0, cols);
    launch(rows, 0);
  } else {
    launch(rows, cols);
  }
  return hipGetLastError();
}

// rows that no group of threads holds in registers (or shorter than a piece):
// dx in two passes over the row, dw and db in strips of rows
template <class XT, class GT, int E>
hipError_t bwd_long(const GT* dy, const XT* x, const uint8_t* xs, const float* w, const float* mean,
                    const float* rstd, int64_t T, int64_t d, GT* dx, float* part, hipStream_t s) {
  if (part) {                                  // before dx, which may overwrite dy
    const Strips st = strips_of(T, d);
    const dim3 grid((unsigned)((d + kColLanes * E - 1) / (kColLanes * E)), (unsigned)st.n);
    ln_bwd_cols<XT, GT, E><<<grid, 256, 0, s>>>(dy, x, xs, mean, rstd, part, T, d, st.rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dx)
    ln_bwd_dx_long<XT, GT, E><<<row_grid(T), 1024, 0, s>>>(dy, x, xs, w, mean, rstd, dx, T, d);
  return hipGetLastError();
}

template <class XT, class GT, int E, bool ODD>
hipError_t bwd(const GT* dy, const XT* x, const uint8_t* xs, const float* w, const float* mean,
               const float* rstd, int64_t T, int64_t d, GT* dx, float* dw, float* db, float* part,
               hipStream_t s) {
  if (bwd_short_fits(T, d))
    return bwd_short<XT, GT, E, ODD>(dy, x, xs, w, mean, rstd, T, d, dx, dw, db, s);
  if (!dw && !db) part = nullptr;
  const BwdPlan p = bwd_plan(T, d, std::is_same_v<XT, kept_t> ? 1024 : 512);
  // the streaming hint needs whole lines
  constexpr bool HINT = !ODD;
  const bool stream = HINT && T * d * (int64_t)(2 * sizeof(GT) + sizeof(XT)) > kStreamBytes;
  hipError_t e;
  if (p.n == 16)
    e = stream ? bwd_rows<XT, GT, E, 16 / E, HINT, ODD>(p, dy, x, xs, w, mean, rstd, T, d, dx,
                                                        part, s)
               : bwd_rows<XT, GT, E, 16 / E, false, ODD>(p, dy, x, xs, w, mean, rstd, T, d, dx,
                                                         part, s);
  else if (p.n)
    e = stream ? bwd_rows<XT, GT, E, 8 / E, HINT, ODD>(p, dy, x, xs, w, mean, rstd, T, d, dx, part,
                                                       s)
               : bwd_rows<XT, GT, E, 8 / E, false, ODD>(p, dy, x, xs, w, mean, rstd, T, d, dx, part,
                                                        s);
  else
    e = bwd_long<XT, GT, ODD ? 1 : E>(dy, x, xs, w, mean, rstd, T, d, dx, part, s);
  if (e != hipSuccess || !part) return e;
  return launch_column_sum(part, p.n ? p.blocks : strips_of(T, d).n, d, 2, dw, db, s);
}

template <class XT, class GT>
hipError_t bwd_by_width(const void* dy, const void* x, const uint8_t* xs, const float* w,
                        const float* mean, const float* rstd, int64_t T, int64_t d, void* dx,
                        float* dw, float* db, float* part, hipStream_t s) {
  const GT* g = (const GT*)dy;
  const XT* v = (const XT*)x;
  constexpr int E = sizeof(XT) + sizeof(GT) <= 4 ? 8 : 4;
  return d % 8 == 0 ? bwd<XT, GT, E, false>(g, v, xs, w, mean, rstd, T, d, (GT*)dx, dw, db, part, s)
                    : bwd<XT, GT, 4, true>(g, v, xs, w, mean, rstd, T, d, (GT*)dx, dw, db, part, s);
}

template <class XT, class YT, int E, int N, bool STREAM, bool ODD>
bool fwd_rows(const XT* x, const float* w, const float* b, int64_t T, int64_t d, float eps, YT* y,
              float* mean, float* rstd, hipStream_t s) {
  const int nt = row_threads(d, N, 1024);
  if (!nt) return false;
  const int G = nt >= 256 ? std::max(1, 512 / nt) : 256 / nt;
  const unsigned grid = (unsigned)std::min<int64_t>((T + G - 1) / G, 1 << 20);
  ln_fwd_rows<XT, YT, E, N / E, STREAM, ODD><<<grid, nt * G, 0, s>>>(x, w, b, y, mean, rstd, T,
                                                                     (int)d, eps, nt);
  return true;
}

// 16 elements a thread, 32 for longer rows (4096 x 13824 bf16: 66 us, 75 with 16)
template <class XT, class YT, int E, bool STREAM, bool ODD>
bool fwd_vec(const XT* x, const float* w, const float* b, int64_t T, int64_t d, float eps, YT* y,
             float* mean, float* rstd, hipStream_t s) {
  return d <= 8192 ? fwd_rows<XT, YT, E, 16, STREAM, ODD>(x, w, b, T, d, eps, y, mean, rstd, s)
                   : fwd_rows<XT, YT, E, 32, STREAM, ODD>(x, w, b, T, d, eps, y, mean, rstd, s);
}

template <class XT, class YT>
hipError_t fwd(const void* xv, const float* w, const float* b, int64_t T, int64_t d, float eps,
               void* yv, float* mean, float* rstd, hipStream_t s) {
  const XT* x = (const XT*)xv;
  YT* y = (YT*)yv;
  bool done;
  if (d % 8 == 0) {
    // elements of a chunk: 4 where the streaming hint or bf16 rows make fp32
    // stores the narrow ones (4096 x 5120 bf16 to fp32 30 us, 34 with 8), else
    // 8 (fp32 to bf16 26 us, 37 with 4; fp32 to fp32 36, 41)
    constexpr bool wide = std::is_same_v<YT, float>;
    constexpr int E = wide && std::is_same_v<XT, __bf16> ? 4 : 8;
    done = T * d * (int64_t)(sizeof(XT) + sizeof(YT)) > kStreamBytes
               ? fwd_vec<XT, YT, wide ? 4 : 8, true, false>(x, w, b, T, d, eps, y, mean, rstd, s)
               : fwd_vec<XT, YT, E, false, false>(x, w, b, T, d, eps, y, mean, rstd, s);
    if (!done)
      ln_fwd_long<XT, YT, 4><<<row_grid(T), 1024, 0, s>>>(x, w, b, y, mean, rstd, T, d, eps);
  } else {
    done = d >= 4 && fwd_vec<XT, YT, 4, false, true>(x, w, b, T, d, eps, y, mean, rstd, s);
    if (!done)
      ln_fwd_long<XT, YT, 1><<<row_grid(T), 1024, 0, s>>>(x, w, b, y, mean, rstd, T, d, eps);
  }
  return hipGetLastError();
}

// out[c] = sum over the P rows of part (row: nout * d floats), in a fixed order:
// 32 columns per workgroup, the rows dealt to 32 lanes, each with eight loads in
// flight (256 x 8192 floats: 4.4 us)
constexpr int kSumCols = 32, kSumLanes = 32;
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part,
                                                          int64_t P, int64_t d, int nout,
                                                          float* __restrict__ out0,
                                                          float* __restrict__ out1) {
  __shared__ float red[kSumLanes][kSumCols + 1];
  const int cl = threadIdx.x % kSumCols, rl = threadIdx.x / kSumCols;
  const int64_t W = d * nout, c = (int64_t)blockIdx.x * kSumCols + cl;
  float a = 0.0f;
  if (c < W) {
    const float* p = part + c;
    int64_t r = rl;
    for (; r + 7 * kSumLanes < P; r += 8 * kSumLanes) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p[(r + k * kSumLanes) * W];
#pragma unroll
      for (int k = 0; k < 8; ++k) a += v[k];
    }
    for (; r < P; r += kSumLanes) a += p[r * W];
  }
  red[rl][cl] = a;
  __syncthreads();
  if (rl == 0 && c < W) {
#pragma unroll
    for (int r = 1; r < kSumLanes; ++r) a += red[r][cl];
    float* o = c < d ? out0 : out1;
    if (o) o[c < d ? c : c - d] = a;
  }
}

}  // namespace

hipError_t launch_column_sum(const float* part, int64_t P, int64_t d, int nout, float* out0,
                             float* out1, hipStream_t s) {
  if (d == 0) return hipSuccess;
  column_sum_kernel<<<(unsigned)((d * nout + kSumCols - 1) / kSumCols), 1024, 0, s>>>(
      part, P, d, nout, out0, out1);
  return hipGetLastError();
}

size_t layer_norm_bwd_ws_bytes(int64_t T, int64_t d) {
  if (bwd_short_fits(T, d)) return 0;
  const BwdPlan p = bwd_plan(T, d);
  return (size_t)(p.n ? p.blocks : strips_of(T, d).n) * 2 * (size_t)d * 4;
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

hipError_t launch_layer_norm_bwd(const void* dy, int gt, const void* x, int xt, const uint8_t* xs,
                                 const float* w, const float* mean, const float* rstd, int64_t T,
                                 int64_t d, void* dx, float* dw, float* db, void* ws,
                                 hipStream_t s) {
  if (T == 0) {
    hipError_t e = dw ? launch_fill_f32(dw, d, 0.0f, s) : hipSuccess;
    if (e != hipSuccess) return e;
    return db ? launch_fill_f32(db, d, 0.0f, s) : hipSuccess;
  }
  float* part = (float*)ws;
  const auto run = [&](auto v, auto g) {
    return bwd_by_width<decltype(v), decltype(g)>(dy, x, xs, w, mean, rstd, T, d, dx, dw, db, part,
                                                  s);
  };
  if (xs) return gt == 0 ? run(kept_t{}, float{}) : run(kept_t{}, __bf16{});
  if (xt == 0) return gt == 0 ? run(float{}, float{}) : run(float{}, __bf16{});
  return gt == 0 ? run(__bf16{}, float{}) : run(__bf16{}, __bf16{});
}

}  // namespace falq
