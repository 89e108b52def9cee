// Softmax cross entropy over the vocabulary of an FP8 output layer, the logits
//   z[t][v] = dec(xq[t]) . dec(wq[v]) / (s_x s_w)
// never kept (of a piece of the vocabulary, the backward's probabilities are):
//   lse[t] = log sum_v exp z[t][v],   loss[t] = lse[t] - z[t][target[t]],
//   dx[t] = dloss[t] sum_v (exp(z[t][v] - lse[t]) - [v = target[t]]) dec(wq[v]) / s_w.
//
// Forward: the product in tiles (linear_act_pipe.hpp, linear_act_tile.hpp), whose
// epilogue leaves of each row the maximum and the sum of exponentials under it over the
// tile's columns, straight from the accumulators, 8 bytes for 64 to 256 logits; a second
// launch joins them.  All of it in float32 and base 2.  The codes are multiplied as
// float16, exactly.  4096 x 32000 x 4096: 747 us, 1.44 PFLOP/s (a library's float16
// product 753), the matrix cores busy 67 % of the cycles at the 1.6 to 1.9 GHz that the
// card's power leaves; 1 token 32 us from a cold cache, W's 131 MB at 4.1 TB/s with the
// launch.  (256 x 256 spills 42 registers, in the loop of the last K steps alone.)
//
// Backward, a piece of the vocabulary after the other: the product again, whose epilogue
// now leaves G = 2^15 (p - [v = target]) of the piece as float16, the target's from its own
// logit, summed in float32, as 2^15 expm1(z - lse): a sure token's gradient is a small
// difference, right down to half a step of lse, a float32 number (2^-21 for an lse of 8 to
// 16); then G times the piece's rows of W, which are read as they lie (F16ByE4M3), added
// onto dx.  2^15 because p may be as small as 1 / V: under it float16 has its full precision
// down to 2^-29 and absolute steps of 2^-39 below, while 1 still fits; E4M3 codes are
// exact in it.  The row's factor dloss / s_w is applied at the end, in float32.
//
// dx in bfloat16, whose half step is 2^-8: the product is FP8's, which of each eight
// products drops what lies 2^-13 below the largest one, so that p is off by expm1 of the sum
// of those (4.5e-5 of the logits' spread with outlier channels: 2^-8 from a spread of a
// hundred on), and G's 11 bits keep the gradient to 2^-11 of its terms.  4096 x 4096 x
// 32000: 1200 to 1280 us, of them G 430 and dx 760 to 820 (1.3 to 1.4 PFLOP/s; the matrix
// cores busy 77 % of the cycles at 1.6 GHz, the power's limit).
//
// dx in float32: the product is the forward's, and G two float16 numbers, itself and what
// that rounding leaves, 2^-22 of the terms; dx's product takes one after the other.  4096 x
// 4096 x 32000: 2480 us where bfloat16 takes 1270.  The gradient as a whole is off by 4e-7
// to 9e-7 (rel-L2; with FP8's logits and one number 1.3e-4 to 1.6e-4).
#include "cross_entropy_plan.hpp"
#include "elem.hpp"
#include "kernels.hpp"
#include "linear_act_pipe.hpp"
#include "linear_act_tile.hpp"

#include <algorithm>

namespace falq {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kGradScale = 32768.0f;

// What the epilogues of the logits take.  V: columns there are (from the piece's
// first on); k: base-2 logits per unit of the accumulators.
struct Logits {
  const float* sx;
  const float* sw;
  const int64_t* target;
  __device__ __forceinline__ float k() const { return kLog2e / (sx[0] * sw[0]); }
};

// over the lanes l, l ^ 32 (and l ^ 16, l ^ 48 with blocks of 16)
template <int BLK>
__device__ __forceinline__ float max_over_g(float v) {
  if constexpr (BLK == 16) v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
template <int BLK>
__device__ __forceinline__ float sum_over_g(float v) {
  if constexpr (BLK == 16) v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// ---- forward --------------------------------------------------------------
// part[i][row] = (maximum, sum of 2^(k (a - maximum))) of the accumulators a of the row's
// columns in the i-th run; at_target[row] = the target's.  Differences of accumulators are
// nearly exact, those of their products with k are off by half a step of a logit: a sure
// token's loss of 0 came out as that, of either sign, and 2^31 and more as infinity.
struct Stats {
  float2* part;
  float* at_target;
};

// (m, s) of two runs
__device__ __forceinline__ void join_runs(float& m, float& s, float m2, float s2, float k) {
  const float top = fmaxf(m, m2);
  // a run without a column is (-inf, 0); one of NaN alone is (-inf, NaN) and stays
  const float a = s == 0.0f ? 0.0f : s * __builtin_amdgcn_exp2f((m - top) * k);
  const float b = s2 == 0.0f ? 0.0f : s2 * __builtin_amdgcn_exp2f((m2 - top) * k);
  m = top;
  s = a + b;
}

template <class C, int MB, int NB, class ACC>
__device__ __forceinline__ void stats_out(uint8_t* smem, const ACC (&acc)[MB][NB], int m0, int n0,
                                          int M, int V, float k, const Logits& lg, const Stats& st,
                                          int tn) {
  // a lane's elements of a block: its row's columns 4 g + (e & 3) + (e >> 2) * SKIP
  constexpr int E = sizeof(ACC) / 4, BLK = E == 4 ? 16 : 32, SKIP = BLK / 4;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wm = w / C::WGN, wn = w % C::WGN;
  const int r = lane % BLK, g = lane / BLK;
  const int col0 = n0 + wn * C::WTN + 4 * g;
  const auto column = [](int j, int e) { return BLK * j + (e & 3) + (e >> 2) * SKIP; };
  const bool whole = n0 + wn * C::WTN + C::WTN <= V;
  float2* const runs = reinterpret_cast<float2*>(smem);      // [WGN][BM]: the waves'
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int row = m0 + wm * C::WTM + i * BLK + r;
    float m = -INFINITY, s = 0.0f;
    if (whole) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) m = fmaxf(m, acc[i][j][e]);
    } else {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (col0 + column(j, e) < V) m = fmaxf(m, acc[i][j][e]);
    }
    m = max_over_g<BLK>(m);
    if (whole) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) s += __builtin_amdgcn_exp2f((acc[i][j][e] - m) * k);
    } else {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (col0 + column(j, e) < V) s += __builtin_amdgcn_exp2f((acc[i][j][e] - m) * k);
    }
    s = sum_over_g<BLK>(s);
    if (g == 0) runs[wn * C::BM + wm * C::WTM + i * BLK + r] = make_float2(m, s);
    // the target's logit, where it is among the wave's columns
    const int64_t t = row < M ? lg.target[row] : -1;
    const int64_t at = t - col0;
    if (t < V && at >= 0 && at < C::WTN) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (at == column(j, e)) st.at_target[row] = acc[i][j][e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < C::BM && m0 + i < M; i += C::kThreads) {
    float2 a = runs[i];
#pragma unroll
    for (int n = 1; n < C::WGN; ++n) {
      const float2 b = runs[n * C::BM + i];
      join_runs(a.x, a.y, b.x, b.y, k);
    }
    st.part[(int64_t)tn * M + m0 + i] = a;
  }
}

template <class C, int PER_CU>
__global__ __launch_bounds__(C::kThreads, PER_CU) void loss_pipe(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, Logits lg, Stats st) {
  int tm, tn;
  gemm::tile_of(gemm::xcd_remap((int)blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = __builtin_amdgcn_readfirstlane(tm * C::BM);
  const int n0 = __builtin_amdgcn_readfirstlane(tn * C::BN);
  pipe_product<E4M3AsF16Wide, C, PER_CU>(
      A, B, M, N, K, m0, n0, 0, INT32_MAX, Exponents{}, [&] { return lg.k(); },
      [&](const auto& acc, float k, uint8_t* smem) {
        stats_out<C>(smem, acc, m0, n0, M, N, k, lg, st, tn);
      });
}
template <class C>
__global__ __launch_bounds__(C::kThreads) void loss_tile(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, Logits lg, Stats st) {
  int tm, tn;
  gemm::tile_of(gemm::xcd_remap((int)blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  tile_product<E4M3AsF16, C>(
      A, B, M, N, K, m0, n0, 0, INT32_MAX, Exponents{}, [&] { return lg.k(); },
      [&](const auto& acc, float k, uint8_t* smem) {
        stats_out<C>(smem, acc, m0, n0, M, N, k, lg, st, tn);
      });
}
// R rows of P runs each per workgroup, the runs dealt to 256 / R lanes in order
template <int R>
__global__ __launch_bounds__(256) void loss_join(const float2* __restrict__ part, int P, int M,
                                                 int64_t V, Logits lg,
                                                 const float* __restrict__ at_target,
                                                 float* __restrict__ loss,
                                                 float* __restrict__ lse) {
  constexpr int L = 256 / R;
  __shared__ float2 red[L][R];
  const int r = threadIdx.x % R, l = threadIdx.x / R;
  const int row = blockIdx.x * R + r;
  const float k = lg.k();
  float m = -INFINITY, s = 0.0f;
  if (row < M)
#pragma unroll 4
    for (int i = l; i < P; i += L) {
      const float2 p = part[(int64_t)i * M + row];
      join_runs(m, s, p.x, p.y, k);
    }
  red[l][r] = make_float2(m, s);
  __syncthreads();
  for (int n = L / 2; n > 0; n /= 2) {
    if (l < n) {
      const float2 p = red[l + n][r];
      join_runs(m, s, p.x, p.y, k);
      red[l][r] = make_float2(m, s);
    }
    __syncthreads();
  }
  if (l != 0 || row >= M) return;
  const float bits = __builtin_amdgcn_logf(s);               // log2
  const int64_t t = lg.target[row];
  if (lse) lse[row] = fmaf(m, k, bits) * kLn2;
  loss[row] = t < 0 ? 0.0f : t >= V ? NAN : fmaf(m - at_target[row], k, bits) * kLn2;
}

// ---- backward -------------------------------------------------------------
// What G's epilogue takes of a row: the logarithm of its terms' factor, 15 - lse in base
// 2 (-inf: the row is not counted, its terms are 0), G at its target and the target (-1:
// none).
struct __attribute__((aligned(16))) GradRow {
  float shift, at_target;
  int target, unused;
};

// a wave a row; G at the target is 2^15 (p - 1)
__global__ __launch_bounds__(256) void grad_rows(const uint8_t* __restrict__ x,
                                                 const uint8_t* __restrict__ w, int M, int d,
                                                 int64_t V, const float* __restrict__ sx,
                                                 const float* __restrict__ sw,
                                                 const int64_t* __restrict__ target,
                                                 const float* __restrict__ lse,
                                                 GradRow* __restrict__ rows) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (row >= M) return;
  const int64_t t = target[row];
  const bool has = t >= 0 && t < V;
  float sum = 0.0f;
  if (has) {
    const uint8_t* a = x + (int64_t)row * d;
    const uint8_t* b = w + t * d;
    for (int i = lane * 16; i < d; i += 1024) {
      const uint4 p = *reinterpret_cast<const uint4*>(a + i);
      const uint4 q = *reinterpret_cast<const uint4*>(b + i);
      const uint32_t u[4] = {p.x, p.y, p.z, p.w}, v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u0 = dec2(u[j], false), u1 = dec2(u[j], true);
        const float2 v0 = dec2(v[j], false), v1 = dec2(v[j], true);
        sum = fmaf(u0.x, v0.x, fmaf(u0.y, v0.y, fmaf(u1.x, v1.x, fmaf(u1.y, v1.y, sum))));
      }
    }
    sum = wave_sum_f32(sum);
  }
  if (lane != 0) return;
  GradRow r;
  r.shift = t < 0 ? -INFINITY : fmaf(lse[row], -kLog2e, 15.0f);
  // (p is 1 at most: half a step of an lse of 10^8 is four.  A NaN stays)
  r.at_target = expm1f(__builtin_elementwise_minimum(sum / (sx[0] * sw[0]) - lse[row], 0.0f)) *
                kGradScale;
  r.target = has ? (int)t : -1;
  r.unused = 0;
  rows[row] = r;
}

// G of a piece, [M x ldg] float16, columns past the vocabulary 0; rest: what that rounding
// leaves of it (null: not wanted)
struct Grads {
  const GradRow* rows;
  _Float16* G;
  _Float16* rest;
  int64_t ldg;
  int v0;              // the piece's first column
};

// through the wave's part of the LDS, as tile_out: eight columns of a row per lane
template <bool REST, class C, int LDS, int MB, int NB, class ACC>
__device__ __forceinline__ void grads_out(uint8_t* smem, const ACC (&acc)[MB][NB], int m0, int n0,
                                          int M, int V, float k, const Grads& gr) {
  const auto row_of = [&](int row) { return gr.rows[row]; };
  const auto out = [&](int row, int col, float(&v)[8], const GradRow& r) {
    typedef _Float16 H8 __attribute__((ext_vector_type(8)));
    H8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], k, r.shift);
    // p is 1 at most, but a logit's error, which goes with its terms and not with lse, may
    // take it past lse, and 2^16 is float16's end.  (minimum: a NaN stays)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_elementwise_minimum(v[i], 15.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_exp2f(v[i]);
    const int at = r.target - gr.v0 - col;
    if ((unsigned)at < 8u) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i == at) v[i] = r.at_target;
    }
    if (col + 8 > V) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i >= V) v[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
    *reinterpret_cast<H8*>(gr.G + (int64_t)row * gr.ldg + col) = h;
    if constexpr (REST) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (_Float16)(v[i] - (float)h[i]);
      *reinterpret_cast<H8*>(gr.rest + (int64_t)row * gr.ldg + col) = h;
    }
  };
  rows_through_lds<C, LDS>(smem, acc, m0, n0, M, (int)gr.ldg, row_of, out);
}

// EXACT: the forward's products, and what G's rounding leaves; otherwise FP8's
template <class C, int PER_CU, bool EXACT>
__global__ __launch_bounds__(C::kThreads, PER_CU) void grads_pipe(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, Logits lg, Grads gr) {
  int tm, tn;
  gemm::tile_of(gemm::xcd_remap((int)blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = __builtin_amdgcn_readfirstlane(tm * C::BM);
  const int n0 = __builtin_amdgcn_readfirstlane(tn * C::BN);
  using OP = std::conditional_t<EXACT, E4M3AsF16Wide, E4M3>;
  pipe_product<OP, C, PER_CU>(
      A, B, M, N, K, m0, n0, 0, INT32_MAX, Exponents{}, [&] { return lg.k(); },
      [&](const auto& acc, float k, uint8_t* smem) {
        grads_out<EXACT, C, Ring<OP, C, PER_CU>::kLds>(smem, acc, m0, n0, M, N, k, gr);
      });
}
template <class C, bool EXACT>
__global__ __launch_bounds__(C::kThreads) void grads_tile(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, Logits lg, Grads gr) {
  int tm, tn;
  gemm::tile_of(gemm::xcd_remap((int)blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  using OP = std::conditional_t<EXACT, E4M3AsF16, E4M3>;
  tile_product<OP, C>(
      A, B, M, N, K, m0, n0, 0, INT32_MAX, Exponents{}, [&] { return lg.k(); },
      [&](const auto& acc, float k, uint8_t* smem) {
        grads_out<EXACT, C, kTileLds<OP, C>>(smem, acc, m0, n0, M, N, k, gr);
      });
}
// dx of all pieces up to this one: sums in `sums` between pieces, dx itself at the last
struct DxOut {
  const int64_t* target;
  const float* dloss;
  const float* sw;
  float* sums;         // [M x N]: read unless this is the first piece
  void* dx;            // [M x N]; null: not the last piece
  int64_t V;
  bool first;
};

// the row's factor, and whether it counts
struct DxRow {
  float factor;
  bool counts;
};
__device__ __forceinline__ DxRow dx_row(const DxOut& o, int row) {
  if (!o.dx) return {1.0f, true};
  const int64_t t = o.target[row];
  return {t >= o.V ? NAN : o.dloss[row] / (o.sw[0] * kGradScale), t >= 0};
}
template <class OT>
__device__ __forceinline__ void dx_out8(float (&v)[8], const DxRow& r, int64_t at,
                                        const DxOut& o) {
  if (!o.first) {
    float t[8];
    load_elems<8>(o.sums + at, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
  }
  if (!o.dx) {
    store_elems<8>(o.sums + at, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r.counts ? v[i] * r.factor : 0.0f;
  store_elems<8>((OT*)o.dx + at, v);
}

// The split and the tile of a workgroup: workgroups go round the eight XCDs, and the
// tiles of a split, which share its columns of G and rows of W, stay on one, whose L2
// then reads them once (where the splits are a multiple of eight).
__device__ __forceinline__ int split_tile(int tilesM, int tilesN, int& tm, int& tn) {
  const int nt = tilesM * tilesN, S = (int)gridDim.x / nt, b = (int)blockIdx.x;
  const int j = S % 8 == 0 ? b / 8 : b;
  const int sp = j / nt + (S % 8 == 0 ? b % 8 * (S / 8) : 0);
  gemm::tile_of(j % nt, tilesM, tilesN, tm, tn);
  return sp;
}

// SPLIT: as linear_act_tile, each split's sums to its plane of `part`
template <class C, int PER_CU, class OT, bool SPLIT>
__global__ __launch_bounds__(C::kThreads, PER_CU) void dx_pipe(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, int rows, DxOut o, float* __restrict__ part, int kc) {
  int tm, tn;
  const int sp = SPLIT ? split_tile(tilesM, tilesN, tm, tn) : 0;
  if constexpr (!SPLIT)
    gemm::tile_of(gemm::xcd_remap((int)blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = __builtin_amdgcn_readfirstlane(tm * C::BM);
  const int n0 = __builtin_amdgcn_readfirstlane(tn * C::BN);
  pipe_product<F16ByE4M3Wide, C, PER_CU>(
      A, B, M, N, K, m0, n0, SPLIT ? sp * kc : 0, SPLIT ? sp * kc + kc : INT32_MAX,
      Exponents{nullptr, nullptr, 0, rows}, [] { return 0; },
      [&](const auto& acc, int, uint8_t* smem) {
        rows_through_lds<C, Ring<F16ByE4M3Wide, C, PER_CU>::kLds>(
            smem, acc, m0, n0, M, N,
            [&](int row) { return SPLIT ? DxRow{} : dx_row(o, row); },
            [&](int row, int col, float(&v)[8], const DxRow& r) {
              if constexpr (SPLIT)
                store_elems<8>(part + ((int64_t)sp * M + row) * N + col, v);
              else
                dx_out8<OT>(v, r, (int64_t)row * N + col, o);
            });
      });
}
// SPLIT: as linear_act_tile, each split's sums to its plane of `part`
template <class C, class OT, bool SPLIT>
__global__ __launch_bounds__(C::kThreads) void dx_tile(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ B, int M, int N, int K, int tilesM,
    int tilesN, int rows, DxOut o, float* __restrict__ part, int kc) {
  int tm, tn;
  const int sp = SPLIT ? split_tile(tilesM, tilesN, tm, tn) : 0;
  if constexpr (!SPLIT)
    gemm::tile_of(gemm::xcd_remap((int)blockIdx.x, tilesM * tilesN), tilesM, tilesN, tm, tn);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  tile_product<F16ByE4M3, C>(
      A, B, M, N, K, m0, n0, SPLIT ? sp * kc : 0, SPLIT ? sp * kc + kc : INT32_MAX,
      Exponents{nullptr, nullptr, 0, rows}, [] { return 0; },
      [&](const auto& acc, int, uint8_t* smem) {
        rows_through_lds<C, kTileLds<F16ByE4M3, C>>(
            smem, acc, m0, n0, M, N,
            [&](int row) { return SPLIT ? DxRow{} : dx_row(o, row); },
            [&](int row, int col, float(&v)[8], const DxRow& r) {
              if constexpr (SPLIT)
                store_elems<8>(part + ((int64_t)sp * M + row) * N + col, v);
              else
                dx_out8<OT>(v, r, (int64_t)row * N + col, o);
            });
      });
}
template <class OT>
__global__ __launch_bounds__(256) void dx_join(const float* __restrict__ part, int S, int64_t M,
                                               int N, DxOut o) {
  const int64_t plane = M * N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < plane / 8;
       i += (int64_t)gridDim.x * 256) {
    const int64_t at = i * 8;
    float v[8];
    load_elems<8>(part + at, v);
    for (int s = 1; s < S; ++s) {
      float t[8];
      load_elems<8>(part + s * plane + at, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    dx_out8<OT>(v, dx_row(o, (int)(at / N)), at, o);
  }
}

// ---- host -----------------------------------------------------------------
using P256 = Tile<256, 256, 2, 2>;
using P256x128 = Tile<256, 128, 2, 2>;
using P192x128 = Tile<192, 128, 2, 2>;
using P128 = Tile<128, 128, 2, 2>;
using T64 = Tile<64, 64, 2, 2, 4>;
using T32 = Tile<32, 64, 1, 4, 4>;

template <class C, int PIPE>
void launch_logits_fwd(const uint8_t* x, const uint8_t* w, int64_t T, int64_t d, int64_t V,
                       const Logits& lg, const Stats& st, hipStream_t s) {
  const int tM = (int)ceil_div64(T, C::BM), tN = (int)ceil_div64(V, C::BN);
  if constexpr (PIPE > 0)
    loss_pipe<C, PIPE><<<tM * tN, C::kThreads, 0, s>>>(x, w, (int)T, (int)V, (int)d, tM, tN, lg,
                                                       st);
  else
    loss_tile<C><<<tM * tN, C::kThreads, 0, s>>>(x, w, (int)T, (int)V, (int)d, tM, tN, lg, st);
}
// V: rows of w from the piece's first on, and columns counted
template <class C, int PIPE, bool EXACT>
void launch_logits_bwd(const uint8_t* x, const uint8_t* w, int64_t T, int64_t d, int64_t V,
                       const Logits& lg, const Grads& gr, hipStream_t s) {
  const int tM = (int)ceil_div64(T, C::BM), tN = (int)ceil_div64(gr.ldg, C::BN);
  if constexpr (PIPE > 0)
    grads_pipe<C, PIPE, EXACT><<<tM * tN, C::kThreads, 0, s>>>(x, w, (int)T, (int)V, (int)d, tM,
                                                               tN, lg, gr);
  else
    grads_tile<C, EXACT><<<tM * tN, C::kThreads, 0, s>>>(x, w, (int)T, (int)V, (int)d, tM, tN, lg,
                                                         gr);
}
void launch_grads(const uint8_t* x, const uint8_t* w, int64_t T, int64_t d, int64_t V,
                  const Logits& lg, const Grads& gr, hipStream_t s) {
  if (gr.rest) {
    switch (loss_kind(T, gr.ldg, d)) {
      case kLoss256: launch_logits_bwd<P256, 1, true>(x, w, T, d, V, lg, gr, s); break;
      case kLoss128: launch_logits_bwd<P128, 2, true>(x, w, T, d, V, lg, gr, s); break;
      case kLoss64: launch_logits_bwd<T64, 0, true>(x, w, T, d, V, lg, gr, s); break;
      default: launch_logits_bwd<T32, 0, true>(x, w, T, d, V, lg, gr, s); break;
    }
    return;
  }
  switch (grad_kind(T, gr.ldg, d)) {
    case kGrad256: launch_logits_bwd<P256, 1, false>(x, w, T, d, V, lg, gr, s); break;
    case kGrad256x128: launch_logits_bwd<P256x128, 2, false>(x, w, T, d, V, lg, gr, s); break;
    case kGrad192x128: launch_logits_bwd<P192x128, 2, false>(x, w, T, d, V, lg, gr, s); break;
    case kGrad128: launch_logits_bwd<P128, 2, false>(x, w, T, d, V, lg, gr, s); break;
    case kGrad64: launch_logits_bwd<T64, 0, false>(x, w, T, d, V, lg, gr, s); break;
    default: launch_logits_bwd<T32, 0, false>(x, w, T, d, V, lg, gr, s); break;
  }
}

template <class C, int PIPE, class OT, bool SPLIT>
void launch_dx(const BwdPlan& p, const uint8_t* g, const uint8_t* w, int64_t T, int64_t d,
               int64_t K, int64_t rows, const DxOut& o, float* part, hipStream_t s) {
  const int tM = (int)ceil_div64(T, C::BM), tN = (int)ceil_div64(d, C::BN);
  if constexpr (PIPE > 0)
    dx_pipe<C, PIPE, OT, SPLIT><<<tM * tN * p.splits, C::kThreads, 0, s>>>(
        g, w, (int)T, (int)d, (int)K, tM, tN, (int)rows, o, part, p.kc);
  else
    dx_tile<C, OT, SPLIT><<<tM * tN * p.splits, C::kThreads, 0, s>>>(
        g, w, (int)T, (int)d, (int)K, tM, tN, (int)rows, o, part, p.kc);
}

template <class OT, bool SPLIT>
void launch_dx_kind(const BwdPlan& p, const uint8_t* g, const uint8_t* w, int64_t T, int64_t d,
                    int64_t K, int64_t rows, const DxOut& o, float* part, hipStream_t s) {
  switch (p.kind) {
    case kDx256:
      if constexpr (!SPLIT) launch_dx<P256, 1, OT, false>(p, g, w, T, d, K, rows, o, part, s);
      break;
    case kDx256x128: launch_dx<P256x128, 2, OT, SPLIT>(p, g, w, T, d, K, rows, o, part, s); break;
    case kDx128: launch_dx<P128, 2, OT, SPLIT>(p, g, w, T, d, K, rows, o, part, s); break;
    case kDx64: launch_dx<T64, 0, OT, SPLIT>(p, g, w, T, d, K, rows, o, part, s); break;
    default: launch_dx<T32, 0, OT, SPLIT>(p, g, w, T, d, K, rows, o, part, s); break;
  }
}

template <class OT>
hipError_t run_dx_product(const BwdPlan& p, const uint8_t* g, const uint8_t* w, int64_t T,
                          int64_t d, int64_t K, int64_t rows, const DxOut& o, float* part,
                          hipStream_t s) {
  if (p.splits == 1) {
    launch_dx_kind<OT, false>(p, g, w, T, d, K, rows, o, part, s);
    return hipGetLastError();
  }
  launch_dx_kind<float, true>(p, g, w, T, d, K, rows, o, part, s);   // sums are float32
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int blocks = (int)std::min<int64_t>((T * d / 8 + 255) / 256, 2048);
  dx_join<OT><<<blocks, 256, 0, s>>>(part, p.splits, T, (int)d, o);
  return hipGetLastError();
}

}  // namespace

// the largest sizes whose tiles, of strips of rows, a grid holds
bool cross_entropy_fits(int64_t T, int64_t d, int64_t V) {
  return T <= (int64_t)1 << 30 && d <= (int64_t)1 << 22 && V <= (int64_t)1 << 22;
}

size_t cross_entropy_fwd_ws_bytes(int64_t T, int64_t d, int64_t V) {
  const int64_t n = strip_of(T);
  // (a strip shorter than the others may have more runs: its tiles may be narrower)
  const int64_t tail = T % kStrip;
  size_t most = 0;
  for (const int64_t m : {n, tail})
    if (m > 0) most = std::max(most, (size_t)(runs_of(m, d, V) * m) * sizeof(float2));
  return T == 0 ? 0 : (size_t)up(n * 4, 256) + most;
}

hipError_t launch_cross_entropy_fwd(const uint8_t* xq, const float* s_x, const uint8_t* wq,
                                    const float* s_w, const int64_t* target, int64_t T, int64_t d,
                                    int64_t V, float* loss, float* lse, void* ws, hipStream_t s) {
  const size_t first = (size_t)up(strip_of(T) * 4, 256);
  for (int64_t r0 = 0; r0 < T; r0 += kStrip) {
    const int64_t n = std::min(kStrip, T - r0);
    const uint8_t* x = xq + r0 * d;
    const Logits lg{s_x, s_w, target + r0};
    const Stats st{(float2*)((char*)ws + first), (float*)ws};
    switch (loss_kind(n, V, d)) {
      case kLoss256: launch_logits_fwd<P256, 1>(x, wq, n, d, V, lg, st, s); break;
      case kLoss128: launch_logits_fwd<P128, 2>(x, wq, n, d, V, lg, st, s); break;
      case kLoss64: launch_logits_fwd<T64, 0>(x, wq, n, d, V, lg, st, s); break;
      default: launch_logits_fwd<T32, 0>(x, wq, n, d, V, lg, st, s); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int P = (int)runs_of(n, d, V);
    float* const out = lse ? lse + r0 : nullptr;
    // few rows a workgroup, so that there are workgroups for all CUs, but 16 where there
    // are: 8-byte partials of adjacent rows are one line
    const auto join = [&](auto rows) {
      constexpr int R = decltype(rows)::value;
      loss_join<R><<<(int)ceil_div64(n, R), 256, 0, s>>>(st.part, P, (int)n, V, lg, st.at_target,
                                                         loss + r0, out);
    };
    if (n < 4 * kCUs)
      join(std::integral_constant<int, 1>{});
    else if (n < 16 * kCUs)
      join(std::integral_constant<int, 4>{});
    else
      join(std::integral_constant<int, 16>{});
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t cross_entropy_bwd_ws_bytes(int64_t T, int64_t d, int64_t V, int dx_type) {
  size_t most = 0;
  for (const int64_t n : {strip_of(T), T % kStrip})
    if (n > 0) most = std::max(most, bwd_plan(n, d, V, dx_type).bytes());
  return most;
}

hipError_t launch_cross_entropy_bwd(const uint8_t* xq, const float* s_x, const uint8_t* wq,
                                    const float* s_w, const int64_t* target, const float* lse,
                                    const float* dloss, int64_t T, int64_t d, int64_t V, void* dx,
                                    int dx_type, void* ws, hipStream_t s) {
  for (int64_t r0 = 0; r0 < T; r0 += kStrip) {
    const int64_t n = std::min(kStrip, T - r0);
    const uint8_t* x = xq + r0 * d;
    const BwdPlan p = bwd_plan(n, d, V, dx_type);
    const Logits lg{s_x, s_w, target + r0};
    uint8_t* const g = (uint8_t*)ws;
    void* const to = (uint8_t*)dx + r0 * d * (dx_type == 0 ? 4 : 2);
    float* const sums = dx_type == 0 ? (float*)to : (float*)(g + p.g);
    float* const part = (float*)(g + p.g + p.sums);
    GradRow* const rows = (GradRow*)(g + p.g + p.sums + p.part);
    grad_rows<<<(unsigned)ceil_div64(n, 4), 256, 0, s>>>(x, wq, (int)n, (int)d, V, s_x, s_w,
                                                         lg.target, lse + r0, rows);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    for (int64_t v0 = 0; v0 < V; v0 += p.width) {
      const int64_t cols = std::min(p.width, V - v0), ld = up(cols, 64);
      const uint8_t* w = wq + v0 * d;
      _Float16* const rest = dx_type == 0 ? (_Float16*)g + n * ld : nullptr;
      launch_grads(x, w, n, d, cols, lg, Grads{rows, (_Float16*)g, rest, ld, (int)v0}, s);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      const bool last = v0 + p.width >= V;
      DxOut o{lg.target, dloss + r0, s_w, sums, last ? to : nullptr, V, v0 == 0};
      if (rest) {                              // G's rounding, and then G, added onto it
        o.dx = nullptr;
        e = run_dx_product<float>(p, (const uint8_t*)rest, w, n, d, ld * 2, cols, o, part, s);
        if (e != hipSuccess) return e;
        o.first = false;
        o.dx = last ? to : nullptr;
        e = run_dx_product<float>(p, g, w, n, d, ld * 2, cols, o, part, s);
      } else {
        e = run_dx_product<__bf16>(p, g, w, n, d, ld * 2, cols, o, part, s);
      }
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace falq
