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

// bias[h, i, j]: bound by its writes (16 x 512 x 512 bf16, 8 MB: 6.8 us traced, a launch's least being 2).  The table's column of a head, laid out by
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
    // (a 64-bit division takes as long as the piece's store)
    int64_t i = n >> 32 ? e / tk : static_cast<uint32_t>(e) / static_cast<uint32_t>(tk), j = e - i * tk;
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

// A wave's sums by relative position in [-most, most], position r in slot
// r + most, and their sums by bucket.  A wave adds to slots of its own with plain
// reads and writes, no two lanes to one slot: LDS atomics took 177 cycles for a
// wave's 64 and have no order.  So that lanes 8 positions apart meet different
// banks, slot n is stored at (n % 8) * (slots / 8) + n / 8.
struct Slots {
  int most, eighth;
  __host__ __device__ __forceinline__ explicit Slots(int m) : most(m), eighth((2 * m + 1 + 7) / 8) {}
  __host__ __device__ __forceinline__ int size() const { return 8 * eighth; }
  __device__ __forceinline__ int at(int rel) const { return (rel + most) % 8 * eighth + (rel + most) / 8; }
};

// store(bucket, sum) for every bucket of the sums of `waves` waves, kept `size()` floats apart; a wave takes every
// waves-th bucket.  All waves have passed a barrier since the sums were written.
template <class F>
__device__ __forceinline__ void bucket_sums(const float* sums, const Slots& slots, int waves, const Buckets& b,
                                            F store) {
  const int l = threadIdx.x % kWave;
  for (int c = threadIdx.x / kWave; c < b.count; c += waves) {
    int from, to;
    b.range(c, slots.most, from, to);
    double s = 0.0;
    for (int r = from + l; r <= to; r += kWave)
      for (int w = 0; w < waves; ++w) s += sums[w * slots.size() + slots.at(r)];
    s = lanes_sum<kWave>(s);
    if (l == 0) store(c, static_cast<float>(s));
  }
}

// Partial sums of dbias by bucket: bound by reading dbias once.  A wave takes a
// row at a time, 16 bytes a lane, and sums it over the batch first.  Pieces that
// lie beyond `reach` on one side have one bucket and stay in a register; the
// others are added to the wave's slots.  8 x 16 x 2048 x 2048 bf16 (1.07 GB) 187 us,
// 5.7 TB/s, with eight batches' loads on their way (four: 210).
template <class Io, bool STREAM>
__global__ __launch_bounds__(kBiasThreads) void relative_bias_bwd_kernel(const typename Io::T* dbias, int64_t sb,
                                                                         int64_t sh, int64_t sq, float* part,
                                                                         int64_t batch, int64_t tq, int64_t tk,
                                                                         int parts, Buckets b) {
  constexpr int V = Io::kVec, kWaves = kBiasThreads / kWave, kDeep = 8;
  FINETUNE_DYNAMIC_LDS(sums);
  const Slots slots(b.reach + V);
  const int h = blockIdx.x / parts, p = blockIdx.x % parts, l = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int64_t rows = (tq + parts - 1) / parts, i0 = p * rows, i1 = i0 + rows < tq ? i0 + rows : tq;
  for (int t = threadIdx.x; t < kWaves * slots.size(); t += kBiasThreads) sums[t] = 0.0f;
  __syncthreads();
  float* mine = sums + wave * slots.size();
  float left = 0.0f, right = 0.0f;
  for (int64_t i = i0 + wave; i < i1; i += kWaves) {
    const typename Io::T* row = dbias + h * sh + i * sq;
    for (int64_t j0 = 0; j0 < tk; j0 += kWave * V) {
      const int64_t j = j0 + l * V;
      float s[V];
#pragma unroll
      for (int x = 0; x < V; ++x) s[x] = 0.0f;
      if (j + V <= tk) {
        for (int64_t n = 0; n < batch; n += kDeep) {  // as many loads on their way
          typename Io::Vec v[kDeep];
#pragma unroll
          for (int m = 0; m < kDeep; ++m) {
            v[m] = typename Io::Vec{};
            if (n + m < batch) v[m] = load_vec<Io, STREAM>(row + (n + m) * sb + j);
          }
#pragma unroll
          for (int m = 0; m < kDeep; ++m)
#pragma unroll
            for (int x = 0; x < V; ++x) s[x] += Io::widen(v[m][x]);
        }
      } else {
        for (int64_t n = 0; n < batch; ++n)
#pragma unroll
          for (int x = 0; x < V; ++x)
            if (j + x < tk) s[x] += Io::widen(row[n * sb + j + x]);
      }
      const int64_t rel = j - i - (tk - tq);
      const bool far = rel <= -b.reach - (V - 1) || rel >= b.reach;
      float all = s[0];
#pragma unroll
      for (int x = 1; x < V; ++x) all += s[x];
      if (far && rel < 0) left += all;
      if (far && rel >= 0) right += all;
      FINETUNE_WAVE_FENCE();
      if (!far && j < tk) {
        float old[V];
#pragma unroll
        for (int x = 0; x < V; ++x) old[x] = mine[slots.at(static_cast<int>(rel) + x)];
#pragma unroll
        for (int x = 0; x < V; ++x) mine[slots.at(static_cast<int>(rel) + x)] = old[x] + s[x];
      }
    }
  }
  left = lanes_sum<kWave>(left);
  right = lanes_sum<kWave>(right);
  FINETUNE_WAVE_FENCE();
  if (l == 0) {
    mine[slots.at(-slots.most)] += left;
    mine[slots.at(slots.most)] += right;
  }
  __syncthreads();
  const int64_t heads = gridDim.x / parts;
  bucket_sums(sums, slots, kWaves, b, [&](int c, float s) { part[(int64_t(c) * heads + h) * parts + p] = s; });
}

}  // namespace finetune
