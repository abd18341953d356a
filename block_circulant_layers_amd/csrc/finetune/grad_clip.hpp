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
constexpr int kClipChunk = 16384;  // elements of one workgroup
constexpr int kClipTensors = 112;  // tensors of one launch (the table travels in the kernel's arguments)

struct ClipTable {
  const void* in[kClipTensors];
  void* out[kClipTensors];
  int64_t count[kClipTensors];
  int first[kClipTensors + 1];  // first chunk of each tensor within the launch
  int8_t dtype[kClipTensors];
  int n;
};
static_assert(sizeof(ClipTable) <= 3800, "kernel arguments are limited to 4 KB");

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

template <class Io>
__device__ __forceinline__ double chunk_square(const void* p, int64_t begin, int64_t end) {
  const auto* g = static_cast<const typename Io::T*>(p);
  double a = 0.0;
  for (int64_t i = begin + threadIdx.x; i < end; i += kClipThreads) {
    const double v = Io::widen(g[i]);
    a += v * v;
  }
  return a;
}

// partial[base + c] = the sum of squares of chunk c
__global__ void __launch_bounds__(kClipThreads) grad_square_kernel(ClipTable t, double* partial) {
  __shared__ double s[kClipThreads / kWave];
  const int c = blockIdx.x, i = tensor_of(t, c);
  const int64_t begin = static_cast<int64_t>(c - t.first[i]) * kClipChunk;
  const int64_t end = begin + kClipChunk < t.count[i] ? begin + kClipChunk : t.count[i];
  double a;
  if (t.dtype[i] == 0)
    a = chunk_square<F32>(t.in[i], begin, end);
  else if (t.dtype[i] == 1)
    a = chunk_square<Bf16>(t.in[i], begin, end);
  else
    a = chunk_square<F16>(t.in[i], begin, end);
  a = block_sum<kClipThreads>(a, s);
  if (threadIdx.x == 0) partial[c] = a;
}

// norm and the factor (factor[0]) from n partial sums, in order
__global__ void __launch_bounds__(kClipThreads)
    grad_norm_kernel(const double* partial, int64_t n, double max_norm, double eps, float* norm, float* factor) {
  __shared__ double s[kClipThreads / kWave];
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kClipThreads) a += partial[i];
  a = sqrt(block_sum<kClipThreads>(a, s));
  if (threadIdx.x == 0) {
    norm[0] = static_cast<float>(a);
    const double f = max_norm / (a + eps);
    if (factor) factor[0] = f > 1.0 ? 1.0f : static_cast<float>(f);
  }
}

template <class Io>
__device__ __forceinline__ void chunk_scale(const void* p, void* q, int64_t begin, int64_t end, float f) {
  const auto* g = static_cast<const typename Io::T*>(p);
  auto* o = static_cast<typename Io::T*>(q);
  for (int64_t i = begin + threadIdx.x; i < end; i += kClipThreads) o[i] = Io::narrow(Io::widen(g[i]) * f);
}

__global__ void __launch_bounds__(kClipThreads) grad_scale_kernel(ClipTable t, const float* factor) {
  const int c = blockIdx.x, i = tensor_of(t, c);
  const float f = factor[0];
  if (f == 1.0f && t.in[i] == t.out[i]) return;  // nothing to change in place
  const int64_t begin = static_cast<int64_t>(c - t.first[i]) * kClipChunk;
  const int64_t end = begin + kClipChunk < t.count[i] ? begin + kClipChunk : t.count[i];
  if (t.dtype[i] == 0)
    chunk_scale<F32>(t.in[i], t.out[i], begin, end, f);
  else if (t.dtype[i] == 1)
    chunk_scale<Bf16>(t.in[i], t.out[i], begin, end, f);
  else
    chunk_scale<F16>(t.in[i], t.out[i], begin, end, f);
}

}  // namespace finetune
