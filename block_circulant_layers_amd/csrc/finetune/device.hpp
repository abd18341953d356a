// device.hpp -- storage types and workgroup reductions of the fine-tuning kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

// The workgroup's LDS block whose size the launch gives.  A host build that
// runs the kernels on CPU threads defines it beforehand.
#ifndef FINETUNE_DYNAMIC_LDS
#define FINETUNE_DYNAMIC_LDS(name) extern __shared__ float name[]
#endif

namespace finetune {

constexpr int kWave = 64;

// Storage types: widened to fp32 on load, rounded to nearest even on store.
// `Vec` is 16 bytes of elements with the alignment of one: rows start at any
// element, and gfx950 loads and stores 16 bytes at any of those addresses.
struct F32 {
  using T = float;
  static constexpr int kVec = 4;
  typedef T Vec __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ float widen(float v) { return v; }
  static __device__ __forceinline__ float narrow(float v) { return v; }
};
struct Bf16 {
  using T = uint16_t;
  static constexpr int kVec = 8;
  typedef T Vec __attribute__((ext_vector_type(8), aligned(2)));
  static __device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }
  static __device__ __forceinline__ uint16_t narrow(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
};
struct F16 {
  using T = uint16_t;
  static constexpr int kVec = 8;
  typedef T Vec __attribute__((ext_vector_type(8), aligned(2)));
  static __device__ __forceinline__ float widen(uint16_t h) {
    return static_cast<float>(__builtin_bit_cast(_Float16, h));
  }
  static __device__ __forceinline__ uint16_t narrow(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  }
};

// Sum of v over the workgroup (NT threads, a multiple of the wave), returned
// to every thread; the order is fixed.  `s` holds NT / 64 slots and may be
// reused after the next barrier.
template <int NT, class V>
__device__ __forceinline__ V block_sum(V v, V* s) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o /= 2) v += __shfl_xor(v, o, kWave);
  if constexpr (NT > kWave) {
    const int w = threadIdx.x / kWave;
    if (threadIdx.x % kWave == 0) s[w] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int i = 1; i < NT / kWave; ++i) v += s[i];
  }
  return v;
}

// The sum over T consecutive threads of a workgroup of NT (T a power of two),
// returned to all of them.  T > 64 takes the workgroup's barrier and T / 64
// slots of `s` per group of T, which may be reused after the next barrier.
template <int T, class V>
__device__ __forceinline__ V group_sum(V v, V* s) {
#pragma unroll
  for (int o = (T < kWave ? T : kWave) / 2; o > 0; o /= 2) v += __shfl_xor(v, o, kWave);
  if constexpr (T > kWave) {
    constexpr int W = T / kWave;
    if (threadIdx.x % kWave == 0) s[threadIdx.x / kWave] = v;
    __syncthreads();
    const V* mine = s + threadIdx.x / T * W;
    v = mine[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v += mine[i];
  }
  return v;
}

}  // namespace finetune
