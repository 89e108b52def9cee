// The product of FP4 operands with a power of two per block of 32 (mx.hpp):
//   z = dec(Xq) dec(Wq)^T + bias,   y = act(z) + residual,
// with the epilogue, the kernels and the rule of linear_act.hip; the matrix core
// applies the blocks' scales itself (v_mfma_scale_f32_16x16x128_f8f6f4 and its form of 32
// x 32 x 64), whose bytes ride along with the codes of a K step, eight for a row.
//
// Bound where it is long by two things: the matrix cores wait for loads and LDS reads, and
// the card's power lowers the clock.  8192 x 8192 x 8192: 250 us (4.4 PFLOP/s; 129 at the
// rate of the instructions alone), the matrix cores busy 58 % of the cycles at 1.7 GHz;
// with zeros for operands busy as much, at 2.2 GHz; 219 without its loads, 220 without its
// LDS reads, 179 without either.  8192 x 11008 x 4096 with gelu and z 227 us, busy 42 % at
// 1.9 GHz: the outputs are 67 at a copy's rate; 1 x 4096 x 4096 4.3 us, 2 TB/s and a launch's
// latency.
#include "activation.hpp"
#include "elem.hpp"
#include "kernels.hpp"
#include "linear_act_pipe.hpp"
#include "linear_act_tile.hpp"
#include "mx_linear_plan.hpp"

#include <algorithm>

namespace falq {
namespace {

// Outputs from what the last-level cache holds on (kStreamBytes) go past the caches: they
// do not fit, and each line written back for another waits.  Alone, and with
// mxfp4_quantize of y behind: 8192 x 11008 x 4096 with gelu and z (361 MB of bfloat16) 227
// and 271 us, 269 and 301 without the hint, 8192 x 8192 x 4096 with gelu and z (256 MiB) 160
// and 200, 169 and 222; 8192 x 11008 x 4096 with gelu and z of float32 280 and 420, 355 and
// 434.  Smaller ones do fit: 8192 x 11008 x 4096 with gelu (180 MB) 219 and 267, 208 and
// 263 without.
template <class C, int PIPE, class OT, bool LEAN = false>
hipError_t mx_tiles(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                    const Epilogue& ep, const Exponents& ex, hipStream_t s) {
  const int tM = (int)((M + C::BM - 1) / C::BM), tN = (int)((N + C::BN - 1) / C::BN);
  if constexpr (PIPE > 0) {
    const auto go = [&](auto stream) {
      linear_act_pipe<Fp4Wide, C, PIPE, OT, decltype(stream)::value, LEAN>
          <<<tM * tN, C::kThreads, 0, s>>>(A, B, (int)M, (int)N, (int)K, tM, tN, ep, ex);
    };
    if (M * N * (int64_t)sizeof(OT) * (1 + (ep.z != nullptr)) >= kStreamBytes)
      go(std::true_type{});
    else
      go(std::false_type{});
  } else {
    linear_act_tile<Fp4, C, OT, false><<<tM * tN, C::kThreads, 0, s>>>(
        A, B, (int)M, (int)N, (int)K, tM, tN, ep, ex);
  }
  return hipGetLastError();
}

template <int MT, int NB, int NW, int U, class OT>
hipError_t mx_few(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                  const Epilogue& ep, const Exponents& ex, hipStream_t s) {
  linear_act_few<Fp4, MT, NB, NW, U, OT>
      <<<(int)((N + NB * 16 - 1) / (NB * 16)), NW * 64, 0, s>>>(A, B, (int)M, (int)N, (int)K, ep,
                                                                ex);
  return hipGetLastError();
}

using T128 = Tile<128, 128, 2, 4, 3>;

template <class OT>
hipError_t mx_by_plan(const uint8_t* A, const uint8_t* B, int64_t M, int64_t N, int64_t K,
                      const Epilogue& ep, const Exponents& ex, float* part, hipStream_t s) {
  const MxPlan p = mx_plan_of(M, N, K);
  if (p.few == 1) return mx_few<1, 1, kFewWaves[1], 1, OT>(A, B, M, N, K, ep, ex, s);
  if (p.few == 2) return mx_few<2, 1, kFewWaves[2], 2, OT>(A, B, M, N, K, ep, ex, s);
  if (p.split > 1) {
    using C = T128;
    const int tM = (int)((M + C::BM - 1) / C::BM), tN = (int)((N + C::BN - 1) / C::BN);
    linear_act_tile<Fp4, C, OT, false, true><<<tM * tN * p.split, C::kThreads, 0, s>>>(
        A, B, (int)M, (int)N, (int)K, tM, tN, ep, ex, part, p.kc);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int blocks = (int)std::min<int64_t>((M * N / 8 + 255) / 256, 2048);
    linear_act_join<Fp4, OT><<<blocks, 256, 0, s>>>(part, p.split, M, (int)N, ep);
    return hipGetLastError();
  }
  switch (p.kind) {
    case kMx256x128: return mx_tiles<Tile<256, 128, 2, 2>, 2, OT, true>(A, B, M, N, K, ep, ex, s);
    case kMx128: return mx_tiles<Tile<128, 128, 2, 2>, 2, OT>(A, B, M, N, K, ep, ex, s);
    case kMx64: return mx_tiles<Tile<64, 64, 2, 2, 4>, 0, OT>(A, B, M, N, K, ep, ex, s);
    default: return mx_tiles<Tile<32, 64, 1, 4, 4>, 0, OT>(A, B, M, N, K, ep, ex, s);
  }
}

}  // namespace

size_t mx_linear_ws_bytes(int64_t T, int64_t d_in, int64_t d_out) {
  if (T == 0 || d_out == 0) return 0;
  const MxPlan p = mx_plan_of(T, d_out, d_in / 2);
  return p.split > 1 ? (size_t)p.split * (size_t)T * (size_t)d_out * 4 : 0;
}

hipError_t launch_mx_linear(const uint8_t* xq, const uint8_t* x_e, const uint8_t* wq,
                            const uint8_t* w_e, const float* bias, const void* residual, int64_t T,
                            int64_t d_in, int64_t d_out, int act, int dtype, void* y, void* z,
                            void* ws, hipStream_t s) {
  if (T == 0 || d_out == 0) return hipSuccess;
  const Epilogue ep{nullptr, nullptr, bias, residual, y, z, act};
  const Exponents ex{x_e, w_e, (int)mx_rows16(T), (int)mx_rows16(d_out)};
  return dtype == 0 ? mx_by_plan<float>(xq, wq, T, d_out, d_in / 2, ep, ex, (float*)ws, s)
                    : mx_by_plan<__bf16>(xq, wq, T, d_out, d_in / 2, ep, ex, (float*)ws, s);
}

}  // namespace falq
