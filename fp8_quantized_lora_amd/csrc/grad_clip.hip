// The global norm of many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over all elements of g^2),  coef = min(1, max_norm / (norm + eps)),
//   g' = g coef.
// Squares are summed in float64 (no overflow below 1e154, no loss over long
// sums; the conversion and the fused multiply-add are far below the memory
// time), in an order that the sizes and the tensors' places within 16 bytes fix.
//
// The tensors' addresses travel in kernel arguments, so a captured graph holds
// them and nothing is copied from the host: up to kTable tensors directly, more
// of them through the workspace, written there by one small launch for each
// kTable tensors, so that the passes over the gradients stay single launches.
//
// Work is counted in chunks of 256 threads x 16 bytes from each tensor's
// address rounded down to 16 bytes: the 16-byte accesses then fit a tensor that
// starts at any element, and only part vectors at its ends are done element by
// element.  Runs of kAhead chunks are dealt round the workgroups (448 tensors of
// 160 M floats 322 us; 338 with one long run for each workgroup), a run's loads
// all in flight.  The second pass goes from the end back: what the first one
// read last is the likeliest to be in the last-level cache still.
//
// Bound by memory: the gradients are read twice (the norm comes before the
// scaling) and written once.  160 M floats: 105 us for the first pass, 215 for
// the second, 6.1 and 6.0 TB/s; a call of a single layer (0.5 M floats) is two
// launches, 6.8 us.
#include "elem.hpp"
#include "kernels.hpp"

#include <algorithm>

namespace falq {
namespace {

constexpr int kTable = 112, kThreads = 256, kAhead = 8;
// elements of a vector and of a chunk
template <class GT>
constexpr int kVec = 16 / sizeof(GT);
template <class GT>
constexpr int kChunk = kThreads * kVec<GT>;
constexpr int kMaxBlocks = 2048;               // eight workgroups per CU

struct Entry {
  const void* g;
  void* out;
  int64_t n;
  uint32_t first;                              // the tensor's first chunk
  int32_t bf16;
};
struct Table {                                 // in the kernel arguments
  Entry e[kTable];
  int count;
  uint32_t chunks;
};
static_assert(sizeof(Table) <= 3600, "kernel arguments");
struct TableInMemory {
  const Entry* e;
  int count;
  uint32_t chunks;
};

__global__ __launch_bounds__(128) void write_table_kernel(Table t, Entry* __restrict__ to) {
  if ((int)threadIdx.x < t.count) to[threadIdx.x] = t.e[threadIdx.x];
}

template <class GT>
__device__ __forceinline__ int lead_of(const GT* g) {
  return (int)((reinterpret_cast<uintptr_t>(g) % 16) / sizeof(GT));
}

// The thread's vectors of chunks [a, b) of a tensor, in order or (BACK) from the
// last to the first: many(i) has kAhead whole vectors at elements i,
// i + kChunk, ...; one(i) a whole vector; each(i) one element of the part
// vectors at the tensor's two ends, which a thread each takes.
template <bool BACK, class GT, class Many, class One, class Each>
__device__ __forceinline__ void run_of(const GT* g, int64_t n, int64_t a, int64_t b, Many&& many,
                                       One&& one, Each&& each) {
  constexpr int V = kVec<GT>;
  const int tid = (int)threadIdx.x;
  const int64_t lead = lead_of(g), mine = (int64_t)tid * V - lead;
  const int64_t head = lead == 0 ? 0 : (V - lead < n ? V - lead : n);
  const int64_t last = (n + lead) / V * V - lead, tail = last > head ? last : head;
  while (a < b) {
    const int64_t first = BACK ? b - kAhead : a;
    if (b - a >= kAhead && first * kChunk<GT> >= lead &&
        (first + kAhead) * kChunk<GT> - lead <= n) {
      many(first * kChunk<GT> + mine);
      (BACK ? b : a) += BACK ? -kAhead : kAhead;
      continue;
    }
    const int64_t c = BACK ? --b : a++, i = c * kChunk<GT> + mine;
    if (i >= 0 && i + V <= n) one(i);
    if (c == 0 && tid < head) each(tid);
    if (tid >= V && tid - V < n - tail && (tail + lead) / kChunk<GT> == c) each(tail + tid - V);
  }
}

// chunks in a workgroup's run: kAhead, fewer where there are not enough for two
// workgroups per CU (4 M floats: 14.9 us, 18.6 with short runs on 2048 workgroups)
__host__ __device__ __forceinline__ uint32_t run_chunks(uint32_t chunks) {
  const uint32_t r = chunks / 512;
  return r < 1 ? 1 : r > kAhead ? kAhead : r;
}

// f(entry, a, b) for the workgroup's runs of chunks, tensor by tensor
template <bool BACK, class Tab, class F>
__device__ __forceinline__ void walk(const Tab& t, F&& f) {
  const uint32_t len = run_chunks(t.chunks), runs = (t.chunks + len - 1) / len;
  for (uint32_t r = blockIdx.x; r < runs; r += gridDim.x) {
    uint32_t c0 = (BACK ? runs - 1 - r : r) * len;
    uint32_t c1 = c0 + len < t.chunks ? c0 + len : t.chunks;
    const uint32_t begin = BACK ? c1 - 1 : c0;
    int k = 0, hi = t.count - 1;               // the tensor of that chunk
    while (k < hi) {
      const int m = (k + hi + 1) / 2;
      if (t.e[m].first <= begin)
        k = m;
      else
        hi = m - 1;
    }
    while (c0 < c1) {
      const uint32_t first = t.e[k].first;
      if (BACK) {
        const uint32_t from = first > c0 ? first : c0;
        f(t.e[k--], (int64_t)(from - first), (int64_t)(c1 - first));
        c1 = from;
      } else {
        const uint32_t end = k + 1 < t.count && t.e[k + 1].first < c1 ? t.e[k + 1].first : c1;
        f(t.e[k++], (int64_t)(c0 - first), (int64_t)(end - first));
        c0 = end;
      }
    }
  }
}

template <class GT>
__device__ __forceinline__ double squares(const GT* g, int64_t n, int64_t a, int64_t b) {
  double s = 0.0;
  auto add = [&](const Raw<GT, kVec<GT>>& v) {
#pragma unroll
    for (int e = 0; e < kVec<GT>; ++e) s = fma((double)v[e], (double)v[e], s);
  };
  run_of<false>(
      g, n, a, b,
      [&](int64_t i) {
        Raw<GT, kVec<GT>> v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v[k].load(g + i + k * kChunk<GT>);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) add(v[k]);
      },
      [&](int64_t i) {
        Raw<GT, kVec<GT>> v;
        v.load(g + i);
        add(v);
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
__device__ __forceinline__ double block_sum_f64(double v) {
  __shared__ double red[kThreads / 64];
  v = wave_sum_f64(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) v += red[i];
  return v;
}

template <class Tab>
__global__ __launch_bounds__(kThreads) void squares_kernel(Tab t, double* __restrict__ part) {
  double s = 0.0;
  walk<false>(t, [&](const Entry& e, int64_t a, int64_t b) {
    s += e.bf16 ? squares((const __bf16*)e.g, e.n, a, b) : squares((const float*)e.g, e.n, a, b);
  });
  s = block_sum_f64(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// the norm from the partial sums, the same in every thread of every workgroup
__device__ __forceinline__ double norm_of(const double* __restrict__ part, int P) {
  double v[kMaxBlocks / kThreads], s = 0.0;
#pragma unroll
  for (int k = 0; k < kMaxBlocks / kThreads; ++k) {
    const int i = k * kThreads + (int)threadIdx.x;
    v[k] = i < P ? part[i] : 0.0;
  }
#pragma unroll
  for (int k = 0; k < kMaxBlocks / kThreads; ++k) s += v[k];
  return sqrt(block_sum_f64(s));
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const double* __restrict__ part, int P,
                                                        float* __restrict__ norm) {
  const double r = norm_of(part, P);
  if (threadIdx.x == 0) *norm = (float)r;
}

template <bool STREAM, class GT>
__device__ __forceinline__ void scale(const GT* g, GT* o, int64_t n, int64_t a, int64_t b,
                                      float c) {
  // the vector form needs the output at the input's place within 16 bytes
  const bool same = lead_of(g) == lead_of(o);
  auto put = [&](int64_t i, const Raw<GT, kVec<GT>>& r) {
    float v[kVec<GT>];
#pragma unroll
    for (int e = 0; e < kVec<GT>; ++e) v[e] = r[e] * c;
    if (same) {
      store_elems<kVec<GT>, STREAM>(o + i, v);
    } else {
#pragma unroll
      for (int e = 0; e < kVec<GT>; ++e) o[i + e] = (GT)v[e];
    }
  };
  run_of<true>(
      g, n, a, b,
      [&](int64_t i) {
        Raw<GT, kVec<GT>> v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v[k].template load<STREAM>(g + i + k * kChunk<GT>);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) put(i + k * kChunk<GT>, v[k]);
      },
      [&](int64_t i) {
        Raw<GT, kVec<GT>> v;
        v.template load<STREAM>(g + i);
        put(i, v);
      },
      [&](int64_t i) { o[i] = (GT)((float)g[i] * c); });
}

// Every workgroup forms the coefficient from the P partial sums (at most 16 KB
// from the caches; a launch between the passes would cost more), and workgroup
// 0 writes the norm.
template <class Tab, bool STREAM>
__global__ __launch_bounds__(kThreads) void scale_kernel(Tab t, const double* __restrict__ part,
                                                         int P, float max_norm, float eps,
                                                         float* __restrict__ norm) {
  const double r = norm_of(part, P);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)r;
  // without a limit, or with nothing but zeros, nothing is scaled, also where the
  // quotient is inf / inf or 0 / 0; a NaN among the elements stays one
  const double to = r + (double)eps;
  const bool free = to == 0.0 || (isinf(max_norm) && !isnan(r));
  float c = free ? 1.0f : (float)((double)max_norm / to);
  c = c > 1.0f ? 1.0f : c;
  walk<true>(t, [&](const Entry& e, int64_t a, int64_t b) {
    if (c == 1.0f && e.g == e.out) return;     // in place and not clipped
    if (e.bf16)
      scale<STREAM>((const __bf16*)e.g, (__bf16*)e.out, e.n, a, b, c);
    else
      scale<STREAM>((const float*)e.g, (float*)e.out, e.n, a, b, c);
  });
}

template <class Tab>
hipError_t passes(const Tab& t, int64_t bytes, float max_norm, float eps, bool clip, float* norm,
                  double* part, hipStream_t s) {
  const uint32_t len = run_chunks(t.chunks);
  const int blocks = (int)std::min<uint32_t>((t.chunks + len - 1) / len, kMaxBlocks);
  if (blocks) squares_kernel<Tab><<<blocks, kThreads, 0, s>>>(t, part);
  if (blocks && clip && 2 * bytes > kStreamBytes)
    scale_kernel<Tab, true><<<blocks, kThreads, 0, s>>>(t, part, blocks, max_norm, eps, norm);
  else if (blocks && clip)
    scale_kernel<Tab, false><<<blocks, kThreads, 0, s>>>(t, part, blocks, max_norm, eps, norm);
  else
    norm_kernel<<<1, kThreads, 0, s>>>(part, blocks, norm);
  return hipGetLastError();
}

}  // namespace

// the partial sums, then the tensors' table where the kernel arguments do not hold it
size_t grad_norm_ws_bytes(int64_t count) {
  return kMaxBlocks * 8 + (count > kTable ? (size_t)count * sizeof(Entry) : 0);
}

hipError_t launch_grad_norm(int64_t count, const void* const* g, const int64_t* n,
                            const int32_t* dtype, float max_norm, float eps, void* const* out,
                            float* norm, void* ws, hipStream_t s) {
  double* part = (double*)ws;
  Entry* table = (Entry*)((uint8_t*)ws + kMaxBlocks * 8);
  Table t;
  t.count = 0;
  t.chunks = 0;
  int64_t bytes = 0;
  int written = 0;
  auto flush = [&] {
    write_table_kernel<<<1, 128, 0, s>>>(t, table + written);
    written += t.count;
    t.count = 0;
    return hipGetLastError();
  };
  for (int64_t i = 0; i < count; ++i) {
    if (n[i] == 0) continue;                   // the entry bounds all elements: chunks fit 32 bits
    if (t.count == kTable) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    const int64_t size = dtype[i] ? 2 : 4, chunk = kThreads * 16 / size;
    const int64_t lead = (int64_t)(reinterpret_cast<uintptr_t>(g[i]) % 16) / size;
    t.e[t.count++] = {g[i], out ? out[i] : nullptr, n[i], t.chunks, dtype[i]};
    bytes += n[i] * size;
    t.chunks += (uint32_t)((n[i] + lead + chunk - 1) / chunk);
  }
  if (!written) return passes(t, bytes, max_norm, eps, out != nullptr, norm, part, s);
  const hipError_t e = flush();
  if (e != hipSuccess) return e;
  return passes(TableInMemory{table, written, t.chunks}, bytes, max_norm, eps, out != nullptr,
                norm, part, s);
}

}  // namespace falq
