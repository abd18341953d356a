// grad_clip.hpp -- the global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over tensors of sum g^2),  out = g min(1, max / (norm + eps)).
//
// Squares and sums run in fp64: an fp32 square overflows from |g| = 1.8e19 on
// and underflows below 1e-23, and the fp64 rate (one multiply-add an element)
// stays far under what the reads leave free.
#pragma once

#include "device.hpp"

namespace finetune {

constexpr int kClipThreads = 256;
constexpr int kClipChunk = 8192;    // elements of one unit of work
constexpr int kClipTensors = 144;   // tensors of one launch (the table travels in the kernel's arguments)
constexpr int kClipGroups = 2048;   // workgroups of a launch at most: 8 a compute unit, and one partial sum each

struct ClipTable {
  const void* in[kClipTensors];
  void* out[kClipTensors];
  int last[kClipTensors];           // elements of each tensor's last chunk; 2 bits of type above them
  int first[kClipTensors + 1];      // first chunk of each tensor within the launch
  int n;
};
static_assert(sizeof(ClipTable) <= 3600, "kernel arguments are limited to 4 KB");
constexpr int kClipTypeShift = 16;
static_assert(kClipChunk < 1 << kClipTypeShift);

// The tensor that chunk c belongs to: the last whose first chunk is <= c.
__device__ __forceinline__ int tensor_of(const ClipTable& t, int c) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// f(storage type, pointer in, pointer out, elements) for chunk c
template <class F>
__device__ __forceinline__ void for_chunk(const ClipTable& t, int c, F f) {
  const int i = tensor_of(t, c), type = t.last[i] >> kClipTypeShift;
  const int64_t begin = static_cast<int64_t>(c - t.first[i]) * kClipChunk;
  const int n = c + 1 == t.first[i + 1] ? t.last[i] & ((1 << kClipTypeShift) - 1) : kClipChunk;
  const auto with = [&](auto io) {
    using T = typename decltype(io)::T;
    f(io, static_cast<const T*>(t.in[i]) + begin, static_cast<T*>(t.out[i]) + begin, n);
  };
  if (type == 0)
    with(F32{});
  else if (type == 1)
    with(Bf16{});
  else
    with(F16{});
}

// partial[workgroup] = the sum of squares of the chunks it walks over
__global__ void __launch_bounds__(kClipThreads) grad_square_kernel(ClipTable t, double* partial) {
  __shared__ double s[kClipThreads / kWave];
  double a[2] = {0.0, 0.0};
  const int chunks = t.first[t.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x)
    for_chunk(t, c, [&](auto io, const auto* g, auto*, int n) {
      using Io = decltype(io);
      constexpr int V = Io::kVec, U = 4;
      const auto add = [&](auto v, int k) {
        const double x = Io::widen(v);
        a[k % 2] = __builtin_fma(x, x, a[k % 2]);
      };
      const Pieces<Io> p(g, 0, n);
      int j = p.first + static_cast<int>(threadIdx.x) * V;
      for (; j + (U - 1) * kClipThreads * V < p.last; j += U * kClipThreads * V) {
        typename Io::Vec raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = load_vec<Io>(g + j + u * kClipThreads * V);
#pragma unroll
        for (int k = 0; k < U * V; ++k) add(raw[k / V][k % V], k);
      }
      for (; j < p.last; j += kClipThreads * V) {
        const typename Io::Vec raw = load_vec<Io>(g + j);
#pragma unroll
        for (int k = 0; k < V; ++k) add(raw[k], k);
      }
      p.template rest<kClipThreads>([&](int i) { add(g[i], 0); });
    });
  const double all = block_sum<kClipThreads>(a[0] + a[1], s);
  if (threadIdx.x == 0) partial[blockIdx.x] = all;
}

// The norm from n partial sums, in a fixed order, in every thread of the workgroup.
__device__ __forceinline__ double norm_of(const double* partial, int64_t n, double* s) {
  double a = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < n; i += kClipThreads) a += partial[i];
  return sqrt(block_sum<kClipThreads>(a, s));
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_kernel(const double* partial, int64_t n, float* norm) {
  __shared__ double s[kClipThreads / kWave];
  const double a = norm_of(partial, n, s);
  if (threadIdx.x == 0) norm[0] = static_cast<float>(a);
}

// out = g min(1, max / (norm + eps)).  Every workgroup sums the partial sums
// itself (16 KB from L2 at most a launch of squares) instead of waiting for a
// kernel that does.  The chunks come in the reverse of the order in which their
// squares were read, so that the last ones read are still in the 256 MB cache.
__global__ void __launch_bounds__(kClipThreads)
    grad_scale_kernel(ClipTable t, const double* partial, int64_t parts, double max_norm, double eps, float* norm) {
  __shared__ double s[kClipThreads / kWave];
  const double a = norm_of(partial, parts, s);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = static_cast<float>(a);
  const double q = max_norm / (a + eps);
  const float f = q > 1.0 ? 1.0f : static_cast<float>(q);
  const int chunks = t.first[t.n];
  for (int c = chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x)
    for_chunk(t, c, [&](auto io, const auto* g, auto* o, int n) {
      using Io = decltype(io);
      constexpr int V = Io::kVec, U = 4;
      if (f == 1.0f && g == o) return;  // nothing to change in place
      const Pieces<Io> p(o, 0, n);
      int j = p.first + static_cast<int>(threadIdx.x) * V;
      const auto scaled = [&](typename Io::Vec v) {
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = Io::narrow(Io::widen(v[k]) * f);
        return v;
      };
      for (; j + (U - 1) * kClipThreads * V < p.last; j += U * kClipThreads * V) {
        typename Io::Vec raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = load_vec<Io>(g + j + u * kClipThreads * V);
#pragma unroll
        for (int u = 0; u < U; ++u) store_vec<Io>(o + j + u * kClipThreads * V, scaled(raw[u]));
      }
      for (; j < p.last; j += kClipThreads * V) store_vec<Io>(o + j, scaled(load_vec<Io>(g + j)));
      p.template rest<kClipThreads>([&](int i) { o[i] = Io::narrow(Io::widen(g[i]) * f); });
    });
}

}  // namespace finetune
