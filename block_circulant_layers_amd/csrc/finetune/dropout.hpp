// dropout.hpp -- dropout whose mask comes from a counter-based generator, with an optional residual sum.
//
// y = residual + (kept ? x * scale : 0), element e kept where its 16 bits of
// Philox4x32-10 are not below a threshold.  One generator call serves the eight
// elements of an aligned group, so a thread takes groups of eight: 16 bytes of
// 16-bit elements, 32 of fp32.  The mask is a function of the element's index
// alone; nothing of it is stored, and the backward computes it again.
//
// Bound by memory: 16384 x 4096 bf16 with a residual moves 403 MB in 65.7 us
// (6.1 TB/s); the generator's twenty wide products for eight elements hide there.
#pragma once

#include "device.hpp"

namespace finetune {

constexpr int kDropThreads = 256;

// Philox4x32-10 (Salmon et al., 2011): ten rounds of two 32 x 32 -> 64 bit products.
struct Philox {
  uint32_t w[4];
  __device__ __forceinline__ Philox(uint64_t block, uint64_t offset, uint64_t seed) {
    uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
    uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
      c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
      c1 = static_cast<uint32_t>(b);
      c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
      c3 = static_cast<uint32_t>(a);
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
  }
  __device__ __forceinline__ uint32_t bits(int i) const { return i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu; }
};

struct DropArgs {
  int64_t rows, d, xs, rs, ys;
  uint64_t seed, offset;
  const uint64_t* device_seed;
  uint32_t least;  // an element is dropped where its bits are below
  float scale;
};

__device__ __forceinline__ uint64_t drop_seed(const DropArgs& a) {
  return a.seed + (a.device_seed ? *a.device_seed : 0);
}

template <class Io, bool RES>
__device__ __forceinline__ float dropped(const DropArgs& a, uint32_t bits, float x, float res) {
  const float kept = bits >= a.least ? x * a.scale : 0.0f;
  return RES ? res + kept : kept;
}

// Tensors without gaps between rows, as one row of n elements.
template <class Io, bool RES, bool STREAM>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(const typename Io::T* x, const typename Io::T* res,
                                                               typename Io::T* y, int64_t n, DropArgs a) {
  using Vec = typename Io::Vec;
  constexpr int V = Io::kVec, P = 8 / V;
  const int64_t step = int64_t(gridDim.x) * kDropThreads, whole = n / 8;
  const uint64_t seed = drop_seed(a);
  for (int64_t g = int64_t(blockIdx.x) * kDropThreads + threadIdx.x; g <= whole; g += step) {
    if (g == whole) {  // the elements after the last group
      const Philox r(static_cast<uint64_t>(g), a.offset, seed);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t e = g * 8 + i;
        if (e < n) y[e] = Io::narrow(dropped<Io, RES>(a, r.bits(i), Io::widen(x[e]), RES ? Io::widen(res[e]) : 0.0f));
      }
      break;
    }
    Vec vx[P], vr[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      vx[p] = load_vec<Io, STREAM>(x + g * 8 + p * V);
      if constexpr (RES) vr[p] = load_vec<Io, STREAM>(res + g * 8 + p * V);
    }
    const Philox r(static_cast<uint64_t>(g), a.offset, seed);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      Vec o;
#pragma unroll
      for (int i = 0; i < V; ++i)
        o[i] = Io::narrow(
            dropped<Io, RES>(a, r.bits(p * V + i), Io::widen(vx[p][i]), RES ? Io::widen(vr[p][i]) : 0.0f));
      store_vec<Io, STREAM>(y + g * 8 + p * V, o);
    }
  }
}

// Rows with gaps: a thread takes the groups of eight of the row-major index, which may span rows.
template <class Io, bool RES>
__global__ __launch_bounds__(kDropThreads) void dropout_rows_kernel(const typename Io::T* x, const typename Io::T* res,
                                                                    typename Io::T* y, DropArgs a) {
  const int64_t n = a.rows * a.d, groups = (n + 7) / 8, step = int64_t(gridDim.x) * kDropThreads;
  const uint64_t seed = drop_seed(a);
  for (int64_t g = int64_t(blockIdx.x) * kDropThreads + threadIdx.x; g < groups; g += step) {
    const Philox r(static_cast<uint64_t>(g), a.offset, seed);
    int64_t row = g * 8 / a.d, col = g * 8 - row * a.d;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (g * 8 + i < n) {
        const float v = Io::widen(x[row * a.xs + col]), s = RES ? Io::widen(res[row * a.rs + col]) : 0.0f;
        y[row * a.ys + col] = Io::narrow(dropped<Io, RES>(a, r.bits(i), v, s));
      }
      if (++col == a.d) col = 0, ++row;
    }
  }
}

}  // namespace finetune
