// Microscaled formats (mx.hpp): FP4 operands quantised and back, and activations
// kept in 8 bits between forward and backward, saved and restored.
//
// Bound by memory, each in one pass: a lane holds eight elements, four lanes a block
// of 32, whose largest magnitude goes round them by cross-lane operands; scaling by a
// power of two is exact, so an element is rounded once, to its code.  8192 x 11008 of
// bfloat16: to FP4 39.5 us (5.8 TB/s), back 34.3, kept in 8 bits 46 (5.9 TB/s), back 48; 11008
// x 4096 of float32 to FP4 31, back to bfloat16 18; one row of 4096 2 to 3.
#include "elem.hpp"
#include "kernels.hpp"
#include "mx.hpp"

#include <algorithm>

namespace falq {
namespace {

typedef v2i v2i_any __attribute__((aligned(1)));

// n of eight elements from p on, the others 0
template <class T>
__device__ __forceinline__ void load_upto8(const T* p, int n, float (&v)[8]) {
  if (n >= 8) {
    load_elems<8>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)p[i] : 0.0f;
  }
}
template <class T>
__device__ __forceinline__ void store_upto8(T* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    store_elems<8>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (T)v[i];
  }
}

// FP4: a workgroup takes 16 rows of one step (256 elements), whose exponent bytes are
// one line of 128; 32 lanes a row, two passes of eight rows.
template <class XT>
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const XT* __restrict__ x,
                                                             uint8_t* __restrict__ q,
                                                             uint8_t* __restrict__ e,
                                                             int64_t rows, int64_t K) {
  const int64_t rows16 = mx_rows16(rows);
  const int l = threadIdx.x & 31, b = l >> 2;
  const int64_t step = blockIdx.x, col = step * kMxStep + l * 8;
  for (int64_t first = (int64_t)blockIdx.y * 16; first < rows; first += (int64_t)gridDim.y * 16) {
    float v[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int64_t row = first + p * 8 + (threadIdx.x >> 5);
      const bool live = row < rows && col < K;               // K is a multiple of 32
      load_upto8(x + (live ? row * K + col : 0), live ? 8 : 0, v[p]);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int64_t row = first + p * 8 + (threadIdx.x >> 5);
      const int ex = mx_exp_fp4(quad_max(mag8(v[p])));
      if (row < rows && col < K)
        *reinterpret_cast<uint32_t*>(q + (row * K + col) / 2) = enc8_fp4(v[p], ex);
      if ((l & 3) == 0) e[mx_scale_at(row, step * 8 + b, rows16)] = (uint8_t)(ex + 127);
    }
  }
}

template <class YT>
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const uint8_t* __restrict__ q,
                                                               const uint8_t* __restrict__ e,
                                                               YT* __restrict__ y, int64_t rows,
                                                               int64_t K) {
  const int64_t rows16 = mx_rows16(rows);
  const int l = threadIdx.x & 31, b = l >> 2;
  const int64_t step = blockIdx.x, col = step * kMxStep + l * 8;
  if (col >= K) return;
#pragma unroll 2
  for (int64_t row = (int64_t)blockIdx.y * 16 + (threadIdx.x >> 5); row < rows;
       row = (row & 8) ? row - 8 + (int64_t)gridDim.y * 16 : row + 8) {
    float v[8];
    dec8_fp4(*reinterpret_cast<const uint32_t*>(q + (row * K + col) / 2),
             e[mx_scale_at(row, step * 8 + b, rows16)], v);
    store_elems<8>(y + row * K + col, v);
  }
}

// 8-bit checkpoints: blocks of 32 along rows of any width, dealt to groups of four
// lanes; a thread's next block is a fixed number of rows and blocks on.
struct Blocks {
  int64_t row, row_by;
  int b, b_by, nb;
  __device__ __forceinline__ Blocks(int64_t nblocks) {
    nb = (int)nblocks;
    const int64_t at = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 4;
    const int64_t by = (int64_t)gridDim.x * blockDim.x / 4;
    row = at / nb;
    b = (int)(at - row * nb);
    row_by = by / nb;
    b_by = (int)(by - row_by * nb);
  }
  __device__ __forceinline__ void next() {
    row += row_by;
    b += b_by;
    if (b >= nb) {
      b -= nb;
      ++row;
    }
  }
};

template <class XT>
__global__ __launch_bounds__(256) void checkpoint_save_kernel(const XT* __restrict__ x,
                                                              uint8_t* __restrict__ q,
                                                              uint8_t* __restrict__ e, int64_t T,
                                                              int64_t d) {
  const int l = threadIdx.x & 3;
  // the four lanes of a block leave together
  for (Blocks k((d + 31) / 32); k.row < T; k.next()) {
    const int64_t col = (int64_t)k.b * 32 + l * 8, at = k.row * d + col;
    const int n = (int)min((int64_t)8, d - col);             // may be 0 or less
    float v[8];
    load_upto8(x + (n > 0 ? at : 0), n, v);
    const int ex = mx_exp_e4m3(quad_max(mag8(v)));
    const float s = exp2_int(-ex);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
    const uint32_t lo = enc4(v[0], v[1], v[2], v[3]), hi = enc4(v[4], v[5], v[6], v[7]);
    if (n >= 8) {
      *reinterpret_cast<v2i_any*>(q + at) = v2i{(int)lo, (int)hi};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) q[at + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
    if (l == 0) e[k.row * k.nb + k.b] = (uint8_t)(ex + 127);
  }
}

template <class YT>
__global__ __launch_bounds__(256) void checkpoint_restore_kernel(const uint8_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ e,
                                                                 YT* __restrict__ y, int64_t T,
                                                                 int64_t d) {
  const int l = threadIdx.x & 3;
  for (Blocks k((d + 31) / 32); k.row < T; k.next()) {
    const int64_t col = (int64_t)k.b * 32 + l * 8, at = k.row * d + col;
    const int n = (int)min((int64_t)8, d - col);
    if (n <= 0) continue;
    const uint32_t s = e[k.row * k.nb + k.b];
    uint32_t w[2] = {0, 0};
    if (n >= 8) {
      const v2i c = *reinterpret_cast<const v2i_any*>(q + at);
      w[0] = (uint32_t)c.x;
      w[1] = (uint32_t)c.y;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 4] |= (uint32_t)q[at + i] << (8 * (i & 3));
    }
    float v[8];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float2 p = dec2_e8m0(w[h / 2], h & 1, s);
      v[2 * h] = p.x;
      v[2 * h + 1] = p.y;
    }
    store_upto8(y + at, n, v);
  }
}

// workgroups of 16 rows of one step each, fewer than 2^24 of 256 threads
dim3 strip_grid(int64_t rows, int64_t K) {
  const int64_t steps = mx_steps(K), most = std::max<int64_t>(1, ((int64_t)1 << 23) / steps);
  return dim3((unsigned)steps,
              (unsigned)std::min<int64_t>({mx_rows16(rows) / 16, most, (int64_t)65535}));
}
// workgroups for blocks of 32
unsigned block_grid(int64_t T, int64_t d) {
  return (unsigned)std::min<int64_t>((T * ((d + 31) / 32) + 63) / 64, 1 << 14);
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, int xt, int64_t rows, int64_t K, uint8_t* q,
                                 uint8_t* e, hipStream_t s) {
  if (rows == 0 || K == 0) return hipSuccess;
  const dim3 grid = strip_grid(rows, K);
  if (xt == 0)
    mxfp4_quantize_kernel<float><<<grid, 256, 0, s>>>((const float*)x, q, e, rows, K);
  else
    mxfp4_quantize_kernel<__bf16><<<grid, 256, 0, s>>>((const __bf16*)x, q, e, rows, K);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* q, const uint8_t* e, int64_t rows, int64_t K,
                                   void* y, int yt, hipStream_t s) {
  if (rows == 0 || K == 0) return hipSuccess;
  const dim3 grid = strip_grid(rows, K);
  if (yt == 0)
    mxfp4_dequantize_kernel<float><<<grid, 256, 0, s>>>(q, e, (float*)y, rows, K);
  else
    mxfp4_dequantize_kernel<__bf16><<<grid, 256, 0, s>>>(q, e, (__bf16*)y, rows, K);
  return hipGetLastError();
}

hipError_t launch_checkpoint_save(const void* x, int xt, int64_t T, int64_t d, uint8_t* q,
                                  uint8_t* e, hipStream_t s) {
  if (T == 0 || d == 0) return hipSuccess;
  const unsigned grid = block_grid(T, d);
  if (xt == 0)
    checkpoint_save_kernel<float><<<grid, 256, 0, s>>>((const float*)x, q, e, T, d);
  else
    checkpoint_save_kernel<__bf16><<<grid, 256, 0, s>>>((const __bf16*)x, q, e, T, d);
  return hipGetLastError();
}

hipError_t launch_checkpoint_restore(const uint8_t* q, const uint8_t* e, int64_t T, int64_t d,
                                     void* y, int yt, hipStream_t s) {
  if (T == 0 || d == 0) return hipSuccess;
  const unsigned grid = block_grid(T, d);
  if (yt == 0)
    checkpoint_restore_kernel<float><<<grid, 256, 0, s>>>(q, e, (float*)y, T, d);
  else
    checkpoint_restore_kernel<__bf16><<<grid, 256, 0, s>>>(q, e, (__bf16*)y, T, d);
  return hipGetLastError();
}

}  // namespace falq
