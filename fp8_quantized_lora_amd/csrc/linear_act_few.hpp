// The epilogue of the FP8 product, and its kernel for few tokens.
#pragma once

#include "activation.hpp"
#include "elem.hpp"
#include "operand_kinds.hpp"

namespace falq {
namespace {

struct Epilogue {
  const float* sa;
  const float* sb;
  const float* bias;        // [N] or null
  const void* residual;     // [M x N] or null; may be y
  void* y;                  // [M x N]
  void* z;                  // [M x N] or null
  int act;
};

// what the products of OP are multiplied by (FP4 operands bring their scales along)
template <class OP>
__device__ __forceinline__ float scale_of(const Epilogue& e) {
  if constexpr (OP::kScaled)
    return 1.0f;
  else
    return 1.0f / (e.sa[0] * e.sb[0]);
}

// E columns of one row
template <int ACT, class OT, bool STREAM, int E>
__device__ __forceinline__ void finish(float (&v)[E], float scale, const float (&bias)[E],
                                       const Epilogue& e, int64_t at) {
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = fmaf(v[i], scale, bias[i]);
  if (e.z) store_elems<E, STREAM>((OT*)e.z + at, v);
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = act_value<ACT, OT>(v[i]);
  if (e.residual) {
    float r[E];
    load_elems<E>((const OT*)e.residual + at, r);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] += r[i];
  }
  store_elems<E, STREAM>((OT*)e.y + at, v);
}

// one column of one row
template <int ACT, class OT>
__device__ __forceinline__ void finish1(float v, float scale, float bias, const Epilogue& e,
                                        int64_t at) {
  float o[1] = {fmaf(v, scale, bias)};
  if (e.z) store_elems<1>((OT*)e.z + at, o);
  o[0] = act_value<ACT, OT>(o[0]);
  if (e.residual) o[0] += (float)((const OT*)e.residual)[at];
  store_elems<1>((OT*)e.y + at, o);
}

template <class OT>
__device__ __forceinline__ void finish1(float v, float scale, float bias, const Epilogue& e,
                                        int64_t at) {
  switch (e.act) {
    case kRelu: return finish1<kRelu, OT>(v, scale, bias, e, at);
    case kGelu: return finish1<kGelu, OT>(v, scale, bias, e, at);
    case kGeluTanh: return finish1<kGeluTanh, OT>(v, scale, bias, e, at);
    case kSilu: return finish1<kSilu, OT>(v, scale, bias, e, at);
    default: return finish1<kNone, OT>(v, scale, bias, e, at);
  }
}

// Few tokens: the weight is read once and everything else is small, so the
// product is a stream over W~.  A workgroup takes 16 NB columns and all of K:
// its NW waves take the 128-byte K steps in turn (adjacent waves read adjacent
// memory), each with the loads of U steps in flight, straight into the
// registers the matrix core reads; the waves' partial sums join in LDS in wave
// order.  A lane holds chunks g and g + 4 (16 bytes each) of row l % 16, g = l / 16,
// of both operands, so whatever order the matrix core takes K in, the operands
// agree.  Chunks past K are cleared in both (a code there may be a NaN).
template <class OP>
__device__ __forceinline__ int few_chunk(int g, int h) {
  if constexpr (OP::kScaled)                                 // the exponents' order
    return OP::chunk(g, h);
  else
    return g + 4 * h;
}
// The sums of a workgroup's columns n0 .. n0 + 16 NB - 1 are left in `part` with a
// barrier behind them: the value of (row, column) is the sum of its NW parts.
template <int MT, int NB, int NW>
using FewParts = float[NW][MT * 16][NB * 16];
template <class OP, int MT, int NB, int NW, int U>
__device__ __forceinline__ void few_product(FewParts<MT, NB, NW>& part,
                                            const uint8_t* __restrict__ A,
                                            const uint8_t* __restrict__ B, int M, int N, int K,
                                            int n0, const Exponents& ex) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int nk = (K + 127) / 128;
  const uint8_t* pa[MT];
  const uint8_t* pb[NB];
#pragma unroll
  for (int m = 0; m < MT; ++m) pa[m] = A + (int64_t)min(m * 16 + r16, M - 1) * K;
#pragma unroll
  for (int n = 0; n < NB; ++n) pb[n] = B + (int64_t)min(n0 + n * 16 + r16, N - 1) * K;
  v4f acc[MT][NB];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  uint4 b[U][NB][2], a[U][MT][2];
  int sb[U][NB], sa[U][MT];
  auto load = [&](int u, int step) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = min(step * 128 + few_chunk<OP>(g, h) * 16, K - 16);
#pragma unroll
      for (int n = 0; n < NB; ++n) b[u][n][h] = *reinterpret_cast<const uint4*>(pb[n] + k);
#pragma unroll
      for (int m = 0; m < MT; ++m) a[u][m][h] = *reinterpret_cast<const uint4*>(pa[m] + k);
    }
    if constexpr (OP::kScaled) {
      const int64_t st = min(step, nk - 1);
#pragma unroll
      for (int n = 0; n < NB; ++n)
        sb[u][n] = *reinterpret_cast<const uint16_t*>(
            ex.b + (st * ex.rows_b + min(n0 + n * 16 + r16, N - 1)) * 8 + 2 * g);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        sa[u][m] = *reinterpret_cast<const uint16_t*>(
            ex.a + (st * ex.rows_a + min(m * 16 + r16, M - 1)) * 8 + 2 * g);
    }
  };
  auto multiply = [&](int u, int step) {
    if (step * 128 + 128 > K) {                              // wave-uniform: behind or across K
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (step * 128 + few_chunk<OP>(g, h) * 16 >= K) {
#pragma unroll
          for (int n = 0; n < NB; ++n) b[u][n][h] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int m = 0; m < MT; ++m) a[u][m][h] = make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n)
        acc[m][n] = OP::mma(OP::make(b[u][n], OP::kScaled ? sb[u][n] : 0),
                            OP::make(a[u][m], OP::kScaled ? sa[u][m] : 0), acc[m][n]);
  };
  if (w < nk) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, w + u * NW);
    int step = w;
    for (; step + U * NW < nk; step += U * NW) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        multiply(u, step + u * NW);
        load(u, step + (U + u) * NW);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(u, step + u * NW);
  }
  // D = B A^T: lane l holds row l % 16 and columns 4 g .. 4 g + 3
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n)
      *reinterpret_cast<v4f*>(&part[w][m * 16 + r16][n * 16 + 4 * g]) = acc[m][n];
  __syncthreads();
}
template <int MT, int NB, int NW>
__device__ __forceinline__ float few_sum(const FewParts<MT, NB, NW>& part, int row, int c) {
  float v = part[0][row][c];
#pragma unroll
  for (int x = 1; x < NW; ++x) v += part[x][row][c];
  return v;
}

template <class OP, int MT, int NB, int NW, int U, class OT>
__global__ __launch_bounds__(NW * 64) void linear_act_few(const uint8_t* __restrict__ A,
                                                          const uint8_t* __restrict__ B, int M,
                                                          int N, int K, Epilogue ep,
                                                          Exponents ex) {
  __shared__ FewParts<MT, NB, NW> part;
  const int n0 = blockIdx.x * NB * 16;
  few_product<OP, MT, NB, NW, U>(part, A, B, M, N, K, n0, ex);
  const float scale = scale_of<OP>(ep);
  for (int i = threadIdx.x; i < M * NB * 16; i += NW * 64) {
    const int row = i / (NB * 16), c = i % (NB * 16), col = n0 + c;
    if (col >= N) continue;
    const float v = few_sum<MT, NB, NW>(part, row, c);
    finish1<OT>(v, scale, ep.bias ? ep.bias[col] : 0.0f, ep, (int64_t)row * N + col);
  }
}

}  // namespace
}  // namespace falq
