// relative_bias.hpp -- a learned bias by buckets of relative positions, and its gradient.
#pragma once

#include "device.hpp"

namespace finetune {

constexpr int kMaxBuckets = 256;    // a side
constexpr int kMaxDistance = 1024;

// The bucket rule as a kernel argument: `first[m]` is the smallest distance
// whose bucket is at least m (first[0] = 0); `reach` = first[side - 1], from
// where on every distance has the last bucket.
struct Buckets {
  int count, side, two_sided, reach;
  int16_t first[kMaxBuckets];

  // the last m with first[m] <= n
  __device__ __forceinline__ int of_distance(int n) const {
    int lo = 0, hi = side;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= n)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  }
  __device__ __forceinline__ int of(int rel) const {
    if (two_sided) return (rel > 0 ? side : 0) + of_distance(rel < 0 ? -rel : rel);
    return of_distance(rel < 0 ? -rel : 0);
  }
  // the relative positions [lo, hi] of bucket c, cut to [-most, most] (lo > hi: none)
  __device__ __forceinline__ void range(int c, int most, int& lo, int& hi) const {
    const bool right = two_sided && c >= side;
    const int m = right ? c - side : c;
    const int a = first[m], b = m + 1 < side ? first[m + 1] - 1 : most;
    if (right) {
      lo = a > 1 ? a : 1, hi = b;
    } else {
      lo = -b, hi = two_sided || m > 0 ? -a : most;
    }
  }
};

constexpr int kBiasThreads = 256;

// bias[h, i, j]: bound by its writes.  The table's column of a head, laid out by
// relative position in [-reach, reach], stays in LDS while a workgroup writes rows
// of that head; positions beyond take the ends.  (grid: heads x row parts)
template <class Io>
__global__ __launch_bounds__(kBiasThreads) void relative_bias_fwd_kernel(const float* table, typename Io::T* bias,
                                                                         int heads, int64_t tq, int64_t tk,
                                                                         int parts, Buckets b) {
  __shared__ float line[2 * kMaxDistance + 1];
  const int h = blockIdx.x / parts, part = blockIdx.x % parts;
  for (int t = threadIdx.x; t < 2 * b.reach + 1; t += kBiasThreads)
    line[t] = table[int64_t(b.of(t - b.reach)) * heads + h];
  __syncthreads();
  const auto value = [&](int64_t rel) {
    const int64_t r = rel < -b.reach ? -b.reach : rel > b.reach ? b.reach : rel;
    return Io::narrow(line[r + b.reach]);
  };
  // the head's tq * tk elements as one row, in 16-byte pieces from the first aligned address on
  typename Io::T* out = bias + h * tq * tk;
  const int64_t n = tq * tk, per = ((n + parts - 1) / parts + Io::kVec - 1) / Io::kVec * Io::kVec;
  const int64_t begin = part * per, end = begin + per < n ? begin + per : n;
  const int64_t off = tk - tq;
  for (int64_t e = begin + int64_t(threadIdx.x) * Io::kVec; e < end; e += kBiasThreads * Io::kVec) {
    int64_t i = e / tk, j = e - i * tk;
    typename Io::Vec v;
#pragma unroll
    for (int c = 0; c < Io::kVec; ++c) {
      v[c] = value(j - i - off);
      if (++j == tk) j = 0, ++i;
    }
    if (e + Io::kVec <= end) {
      store_vec<Io>(out + e, v);
    } else {
      for (int c = 0; c < Io::kVec; ++c)
        if (e + c < end) out[e + c] = v[c];
    }
  }
}

// Partial sums of dbias by relative position: a workgroup takes `rows` rows of a
// head's matrix over the whole batch; a thread owns columns of the rows' skewed
// layout... one relative position a thread, cut to [-reach, reach], so that no two
// threads add to the same place and the order is fixed.
template <class Io>
__global__ __launch_bounds__(kBiasThreads) void relative_bias_bwd_kernel(const typename Io::T* dbias, int64_t sb,
                                                                         int64_t sh, int64_t sq, float* part,
                                                                         int64_t batch, int64_t tq, int64_t tk,
                                                                         int parts, Buckets b) {
  __shared__ float sums[kBiasThreads];
  __shared__ double total[2 * kMaxBuckets];
  const int h = blockIdx.x / parts, p = blockIdx.x % parts;
  const int64_t rows = (tq + parts - 1) / parts, i0 = p * rows, i1 = i0 + rows < tq ? i0 + rows : tq;
  for (int t = threadIdx.x; t < b.count; t += kBiasThreads) total[t] = 0.0;
  const int64_t off = tk - tq;
  // relative positions of these rows: [-(i1 - 1) - off, tk - 1 - i0 - off], a block of threads at a time
  const int64_t lo = -(i1 - 1) - off, hi = tk - 1 - i0 - off;
  for (int64_t r0 = lo; r0 <= hi && i1 > i0; r0 += kBiasThreads) {
    const int64_t rel = r0 + threadIdx.x;
    float s = 0.0f;
    if (rel <= hi)
      for (int64_t n = 0; n < batch; ++n)
        for (int64_t i = i0; i < i1; ++i) {
          const int64_t j = rel + i + off;
          if (j >= 0 && j < tk) s += Io::widen(dbias[n * sb + h * sh + i * sq + j]);
        }
    __syncthreads();
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int c = threadIdx.x; c < b.count; c += kBiasThreads) {
      int from, to;
      b.range(c, 1 << 30, from, to);
      double d = 0.0;
      for (int64_t x = from > r0 ? from : r0; x <= to && x < r0 + kBiasThreads; ++x) d += sums[x - r0];
      total[c] += d;
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < b.count; c += kBiasThreads)
    part[(int64_t(c) * (gridDim.x / parts) + h) * parts + p] = static_cast<float>(total[c]);
}

}  // namespace finetune
