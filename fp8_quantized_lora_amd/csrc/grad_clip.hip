// The global norm of many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over all elements of g^2),  coef = min(1, max_norm / (norm + eps)),
//   g' = g coef.
// Squares are summed in float64 (no overflow below 1e154, no loss over long
// sums; the conversion and the fused multiply-add are far below the memory
// time), in an order that the sizes fix.
//
// The tensors' addresses travel in the kernel arguments, kTable of them per
// launch, so a captured graph holds them and nothing is copied to the device.
// Work is dealt in chunks of kChunk elements, counted from each tensor's
// address rounded down to 16 bytes: the 16-byte accesses then fit a tensor
// that starts at any element, and only its first and last vectors are done
// element by element.
#include "elem.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace falq {
namespace {

constexpr int kTable = 112;                    // 112 * 32 + 8 bytes of kernel arguments
constexpr int kChunk = 8192, kThreads = 256, kMaxBlocks = 1024;

struct Table {
  const void* g[kTable];
  void* out[kTable];
  int64_t n[kTable];
  uint32_t first[kTable];                      // the tensor's first chunk
  uint32_t bf16[(kTable + 31) / 32];           // its type
  int count;
  uint32_t chunks;
};
static_assert(sizeof(Table) <= 3800, "kernel arguments");

template <class GT>
__device__ __forceinline__ int lead_of(const GT* g) {
  return (int)((reinterpret_cast<uintptr_t>(g) % 16) / sizeof(GT));
}

// f(i, v): vectors of 8 elements from element i on (all inside); f1(i): one element
template <class GT, class F, class F1>
__device__ __forceinline__ void each(const GT* g, int64_t n, uint32_t chunk, F&& f, F1&& f1) {
  const int lead = lead_of(g);
  const int64_t base = (int64_t)chunk * kChunk - lead;
#pragma unroll 4
  for (int k = 0; k < kChunk / (kThreads * 8); ++k) {
    const int64_t i = base + (k * kThreads + (int)threadIdx.x) * 8;
    if (i >= 0 && i + 8 <= n) {
      f(i);
    } else if (i + 8 > 0 && i < n) {
      for (int64_t j = i < 0 ? 0 : i; j < (i + 8 < n ? i + 8 : n); ++j) f1(j);
    }
  }
}

__device__ __forceinline__ int tensor_of(const Table& t, uint32_t chunk) {
  int lo = 0, hi = t.count - 1;                // the last tensor whose first chunk is <= chunk
  while (lo < hi) {
    const int m = (lo + hi + 1) / 2;
    if (t.first[m] <= chunk)
      lo = m;
    else
      hi = m - 1;
  }
  return lo;
}

template <class GT>
__device__ __forceinline__ double chunk_squares(const GT* g, int64_t n, uint32_t chunk) {
  double s = 0.0;
  each(
      g, n, chunk,
      [&](int64_t i) {
        float v[8];
        load_elems<8>(g + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fma((double)v[e], (double)v[e], s);
      },
      [&](int64_t i) { s = fma((double)(float)g[i], (double)(float)g[i], s); });
  return s;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// sum over the workgroup, in every thread
template <int NT>
__device__ __forceinline__ double block_sum_f64(double v) {
  __shared__ double red[NT / 64];
  v = wave_sum_f64(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) v += red[i];
  return v;
}

__global__ __launch_bounds__(kThreads) void squares_kernel(Table t, double* __restrict__ part) {
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const uint32_t in = c - t.first[k];
    if ((t.bf16[k / 32] >> (k % 32)) & 1)
      s += chunk_squares((const __bf16*)t.g[k], t.n[k], in);
    else
      s += chunk_squares((const float*)t.g[k], t.n[k], in);
  }
  s = block_sum_f64<kThreads>(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// norm (and the coefficient) from the partial sums, in one workgroup
__global__ __launch_bounds__(kThreads) void norm_kernel(const double* __restrict__ part, int P,
                                                        float max_norm, float eps,
                                                        float* __restrict__ norm,
                                                        float* __restrict__ coef) {
  double s = 0.0;
  for (int i = threadIdx.x; i < P; i += kThreads) s += part[i];
  const double r = sqrt(block_sum_f64<kThreads>(s));
  if (threadIdx.x == 0) {
    if (norm) *norm = (float)r;
    if (coef) {
      const float c = (float)((double)max_norm / (r + (double)eps));
      *coef = c > 1.0f ? 1.0f : c;             // NaN stays NaN
    }
  }
}

template <class GT>
__device__ __forceinline__ void chunk_scale(const GT* g, GT* o, int64_t n, uint32_t chunk,
                                            float c) {
  // the vector form needs the output at the input's place within 16 bytes
  const bool same = lead_of(g) == lead_of(o);
  each(
      g, n, chunk,
      [&](int64_t i) {
        float v[8];
        load_elems<8>(g + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= c;
        if (same) {
          store_elems<8>(o + i, v);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[i + e] = (GT)v[e];
        }
      },
      [&](int64_t i) { o[i] = (GT)((float)g[i] * c); });
}

__global__ __launch_bounds__(kThreads) void scale_kernel(Table t, const float* __restrict__ coef) {
  const float c = *coef;
  for (uint32_t b = blockIdx.x; b < t.chunks; b += gridDim.x) {
    const int k = tensor_of(t, b);
    if (c == 1.0f && t.g[k] == t.out[k]) continue;           // in place and not clipped
    const uint32_t in = b - t.first[k];
    if ((t.bf16[k / 32] >> (k % 32)) & 1)
      chunk_scale((const __bf16*)t.g[k], (__bf16*)t.out[k], t.n[k], in, c);
    else
      chunk_scale((const float*)t.g[k], (float*)t.out[k], t.n[k], in, c);
  }
}

// calls f(table, blocks) for each table of tensors; empty tensors are left out
// (the entry bounds the elements of all tensors, so the chunks fit 32 bits)
template <class F>
hipError_t each_table(int64_t count, const void* const* g, const int64_t* n, const int32_t* dtype,
                      void* const* out, F&& f) {
  int64_t i = 0;
  while (i < count) {
    Table t;
    t.count = 0;
    for (uint32_t& w : t.bf16) w = 0;
    uint64_t chunks = 0;
    for (; i < count && t.count < kTable; ++i) {
      if (n[i] == 0) continue;
      const int k = t.count;
      const int size = dtype[i] ? 2 : 4;
      const int64_t lead = (int64_t)(reinterpret_cast<uintptr_t>(g[i]) % 16) / size;
      const uint64_t c = (uint64_t)((n[i] + lead + kChunk - 1) / kChunk);
      t.g[k] = g[i];
      t.out[k] = out ? out[i] : nullptr;
      t.n[k] = n[i];
      t.first[k] = (uint32_t)chunks;
      if (dtype[i]) t.bf16[k / 32] |= 1u << (k % 32);
      chunks += c;
      ++t.count;
    }
    if (t.count == 0) break;
    t.chunks = (uint32_t)chunks;
    const hipError_t e = f(t, (int)std::min<uint64_t>(chunks, kMaxBlocks));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// the coefficient, then kMaxBlocks partial sums per table
size_t grad_norm_ws_bytes(int64_t count) {
  return 64 + (size_t)((count + kTable - 1) / kTable) * kMaxBlocks * 8;
}

hipError_t launch_grad_norm(int64_t count, const void* const* g, const int64_t* n,
                            const int32_t* dtype, float max_norm, float eps, void* const* out,
                            float* norm, void* ws, hipStream_t s) {
  float* coef = (float*)ws;
  double* part = (double*)((uint8_t*)ws + 64);
  int P = 0;
  hipError_t e = each_table(count, g, n, dtype, out, [&](const Table& t, int blocks) {
    squares_kernel<<<blocks, kThreads, 0, s>>>(t, part + P);
    P += blocks;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  norm_kernel<<<1, kThreads, 0, s>>>(part, P, max_norm, eps, norm, out ? coef : nullptr);
  e = hipGetLastError();
  if (e != hipSuccess || !out) return e;
  return each_table(count, g, n, dtype, out, [&](const Table& t, int blocks) {
    scale_kernel<<<std::min<int>(t.chunks, 4 * blocks), kThreads, 0, s>>>(t, coef);
    return hipGetLastError();
  });
}

}  // namespace falq
