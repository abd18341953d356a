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
constexpr int kClipChunk = 4096;    // elements of one unit of work
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

// This workgroup's share of the launch: consecutive chunks, as one run a tensor
// they touch.  f(storage type, pointer in, pointer out, elements) for every run,
// the last one first if BACK.  (Single chunks dealt out in turn took 533 us where
// runs take TBD us: every chunk waited for its table entries.)
template <bool BACK, class F>
__device__ __forceinline__ void for_runs(const ClipTable& t, F f) {
  const int chunks = t.first[t.n], per = (chunks + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  int c0 = static_cast<int>(blockIdx.x) * per, c1 = c0 + per < chunks ? c0 + per : chunks;
  if (c0 >= c1) return;
  for (int i = tensor_of(t, BACK ? c1 - 1 : c0); c0 < c1; i += BACK ? -1 : 1) {
    const int from = t.first[i], to = t.first[i + 1], last = t.last[i];
    const int a = from > c0 ? from : c0, b = to < c1 ? to : c1;
    const int64_t begin = static_cast<int64_t>(a - from) * kClipChunk;
    const int n = (b - a) * kClipChunk - (b == to ? kClipChunk - (last & ((1 << kClipTypeShift) - 1)) : 0);
    const auto with = [&](auto io) {
      using T = typename decltype(io)::T;
      f(io, static_cast<const T*>(t.in[i]) + begin, static_cast<T*>(t.out[i]) + begin, n);
    };
    const int type = last >> kClipTypeShift;
    if (type == 0)
      with(F32{});
    else if (type == 1)
      with(Bf16{});
    else
      with(F16{});
    if (BACK)
      c1 = a;
    else
      c0 = b;
  }
}

// g(column, piece or single value) over n elements at p: batches of U pieces a
// thread, the last batch first if BACK
template <class Io, int U, bool BACK, class Batch, class Piece, class One>
__device__ __forceinline__ void for_pieces(const typename Io::T* at, int n, Batch batch, Piece piece, One one) {
  constexpr int V = Io::kVec, STEP = U * kClipThreads * V;
  const Pieces<Io> p(at, 0, n);
  const int t = p.first + static_cast<int>(threadIdx.x) * V, full = (p.last - p.first) / STEP;
  const auto rest = [&]() {
    for (int j = t + full * STEP; j < p.last; j += kClipThreads * V) piece(j);
    p.template rest<kClipThreads>(one);
  };
  if (BACK) rest();
  for (int k = 0; k < full; ++k) batch(t + (BACK ? full - 1 - k : k) * STEP);
  if (!BACK) rest();
}

// partial[workgroup] = the sum of squares of the chunks it walks over
__global__ void __launch_bounds__(kClipThreads) grad_square_kernel(ClipTable t, double* partial) {
  __shared__ double s[kClipThreads / kWave];
  double a[2] = {0.0, 0.0};
  for_runs<false>(t, [&](auto io, const auto* g, auto*, int n) {
    using Io = decltype(io);
    constexpr int V = Io::kVec, U = 8;
    const auto add = [&](auto v, int k) {
      const double x = Io::widen(v);
      a[k % 2] = __builtin_fma(x, x, a[k % 2]);
    };
    for_pieces<Io, U, false>(
        g, n,
        [&](int j) {
          typename Io::Vec raw[U];
#pragma unroll
          for (int u = 0; u < U; ++u) raw[u] = load_vec<Io>(g + j + u * kClipThreads * V);
#pragma unroll
          for (int k = 0; k < U * V; ++k) add(raw[k / V][k % V], k);
        },
        [&](int j) {
          const typename Io::Vec raw = load_vec<Io>(g + j);
#pragma unroll
          for (int k = 0; k < V; ++k) add(raw[k], k);
        },
        [&](int i) { add(g[i], 0); });
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
// kernel that does, and goes through its share backwards: what the squares
// read last is still in the 256 MB cache.
__global__ void __launch_bounds__(kClipThreads)
    grad_scale_kernel(ClipTable t, const double* partial, int64_t parts, double max_norm, double eps, float* norm) {
  __shared__ double s[kClipThreads / kWave];
  const double a = norm_of(partial, parts, s);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = static_cast<float>(a);
  const double q = max_norm / (a + eps);
  const float f = q > 1.0 ? 1.0f : static_cast<float>(q);
  for_runs<true>(t, [&](auto io, const auto* g, auto* o, int n) {
    using Io = decltype(io);
    constexpr int V = Io::kVec, U = 4;
    if (f == 1.0f && g == o) return;  // nothing to change in place
    const auto scaled = [&](typename Io::Vec v) {
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = Io::narrow(Io::widen(v[k]) * f);
      return v;
    };
    for_pieces<Io, U, true>(
        o, n,
        [&](int j) {
          typename Io::Vec raw[U];
#pragma unroll
          for (int u = 0; u < U; ++u) raw[u] = load_vec<Io>(g + j + u * kClipThreads * V);
#pragma unroll
          for (int u = 0; u < U; ++u) store_vec<Io>(o + j + u * kClipThreads * V, scaled(raw[u]));
        },
        [&](int j) { store_vec<Io>(o + j, scaled(load_vec<Io>(g + j))); },
        [&](int i) { o[i] = Io::narrow(Io::widen(g[i]) * f); });
  });
}

}  // namespace finetune
