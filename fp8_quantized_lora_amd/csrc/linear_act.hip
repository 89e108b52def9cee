// The FP8 product of a melded linear layer with its epilogue:
//   z = dec(X~) dec(W~)^T / (s_x s_w) + bias,   y = act(z) + residual,
// y, z and residual all bfloat16 or all float32; z is written where the
// caller keeps it for the backward.  Accumulation, bias, activation and
// residual are float32, and each output is rounded once.
//
// Two kinds of tile kernel, for any tile size and any K that is a multiple of 16
// (in a last step of fewer than 128 bytes the chunks past K are cleared in LDS),
// both with v_mfma_f32_16x16x128_f8f6f4 on swizzled rows of 128 K-bytes that were
// loaded straight into LDS: linear_act_pipe (linear_act_pipe.hpp) for many
// outputs, linear_act_tile (linear_act_tile.hpp) for few.
//
// Long products are bound by the matrix cores, in part by their power, and by
// the outputs (8192 x 11008 x 4096 with gelu and z: 305 to 316 us, 2.4 PFLOP/s; 275
// without the epilogue's work and z; 4096 x 5120 x 13824 with a residual 201 to 213
// us, 2.8 PFLOP/s), few tokens by reading W~ (1 x 4096 x 4096: 5.2 us on the GPU, 3.2
// TB/s, of which a launch's latency is half).
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
#include "linear_act_pipe.hpp"
#include "linear_act_plan.hpp"
#include "linear_act_tile.hpp"

#include <algorithm>

namespace falq {
namespace {

// Outputs above this go past the caches, which keeps the operands in them.
// Below, the hint only moves the cost to the reader: with fp8_quantize of y
// behind the product, 8192 x 11008 x 4096 gelu (172 MB) 417 us with it, 425
// without (alone 306 and 335); 4096 x 8192 x 4096 (64 MB) 140 and 135.
constexpr int64_t kStreamOut = (int64_t)80 << 20;

// whether the outputs take the streaming hint, which needs whole lines: 16-byte
// stores, so bfloat16
template <class OT>
bool stream_outputs(int64_t M, int64_t N, const Epilogue& ep) {
  return sizeof(OT) == 2 && M * N * 2 * (1 + (ep.z != nullptr)) > kStreamOut;
}

// tiles of C: linear_act_tile, or PIPE workgroups of linear_act_pipe per CU.  MANY:
// the rule takes them for outputs that are streamed, too.
template <class C, int PIPE, class OT, bool MANY = true>
hipError_t launch_tiles(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                        const Epilogue& ep, hipStream_t s) {
  const int tM = (int)((M + C::BM - 1) / C::BM), tN = (int)((N + C::BN - 1) / C::BN);
  const auto go = [&](auto stream) {
    constexpr bool STREAM = decltype(stream)::value;
    if constexpr (PIPE > 0)
      linear_act_pipe<C, PIPE, OT, STREAM><<<tM * tN, C::kThreads, 0, s>>>(
          A, B, (int)M, (int)N, (int)K, tM, tN, ep);
    else
      linear_act_tile<C, OT, STREAM><<<tM * tN, C::kThreads, 0, s>>>(A, B, (int)M, (int)N, (int)K,
                                                                     tM, tN, ep);
  };
  if (MANY && stream_outputs<OT>(M, N, ep))
    go(std::bool_constant<MANY && sizeof(OT) == 2>{});
  else
    go(std::false_type{});
  return hipGetLastError();
}

template <int MT, int NB, int NW, int U, class OT>
hipError_t launch_few(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                      const Epilogue& ep, hipStream_t s) {
  linear_act_few<MT, NB, NW, U, OT><<<(int)((N + NB * 16 - 1) / (NB * 16)), NW * 64, 0, s>>>(
      A, B, (int)M, (int)N, (int)K, ep);
  return hipGetLastError();
}

using T128 = Tile<128, 128, 2, 4, 3>;

template <class OT>
hipError_t launch_kind(TileKind k, const uint8_t* A, const uint8_t* B, int64_t M, int64_t N,
                       int64_t K, const Epilogue& ep, hipStream_t s) {
  switch (k) {
    case k256x320: return launch_tiles<Tile<256, 320, 2, 2>, 1, OT>(A, B, M, N, K, ep, s);
    case k256: return launch_tiles<Tile<256, 256, 2, 2>, 1, OT>(A, B, M, N, K, ep, s);
    case k256x128: return launch_tiles<Tile<256, 128, 2, 2>, 2, OT>(A, B, M, N, K, ep, s);
    case k128x256: return launch_tiles<Tile<128, 256, 2, 2>, 2, OT>(A, B, M, N, K, ep, s);
    case k192x128: return launch_tiles<Tile<192, 128, 2, 2>, 2, OT>(A, B, M, N, K, ep, s);
    case k128x192w8: return launch_tiles<Tile<128, 192, 2, 4, 3>, 0, OT>(A, B, M, N, K, ep, s);
    case k128: return launch_tiles<Tile<128, 128, 2, 2>, 2, OT>(A, B, M, N, K, ep, s);
    case k128w8: return launch_tiles<T128, 0, OT, false>(A, B, M, N, K, ep, s);
    case k64: return launch_tiles<Tile<64, 64, 2, 2, 4>, 0, OT>(A, B, M, N, K, ep, s);
    default: return launch_tiles<Tile<32, 64, 1, 4, 4>, 0, OT>(A, B, M, N, K, ep, s);
  }
}

template <class OT>
hipError_t launch_split(const Plan& p, const uint8_t* A, const uint8_t* B, int64_t M, int64_t N,
                        int64_t K, const Epilogue& ep, float* part, hipStream_t s) {
  using C = T128;
  const int tM = (int)((M + C::BM - 1) / C::BM), tN = (int)((N + C::BN - 1) / C::BN);
  linear_act_tile<C, OT, false, true><<<tM * tN * p.split, C::kThreads, 0, s>>>(
      A, B, (int)M, (int)N, (int)K, tM, tN, ep, part, p.kc);
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
  if (p.few == 1) return launch_few<1, 1, kFewWaves[1], 1, OT>(A, B, M, N, K, ep, s);
  if (p.few == 2) return launch_few<2, 1, kFewWaves[2], 2, OT>(A, B, M, N, K, ep, s);
  if (p.split > 1) return launch_split<OT>(p, A, B, M, N, K, ep, part, s);
  return launch_kind<OT>(p.kind, A, B, M, N, K, ep, s);
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
