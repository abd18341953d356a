// device.hpp -- storage types and workgroup reductions of the fine-tuning kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

// The workgroup's LDS block whose size the launch gives.  A host build that
// runs the kernels on CPU threads defines it beforehand.
#ifndef FINETUNE_DYNAMIC_LDS
#define FINETUNE_DYNAMIC_LDS(name) extern __shared__ float name[]
#endif

// Two pieces of gfx950 assembly, which a host build defines otherwise: the
// maximum of three values (the compiler's fmaxf first quiets every operand;
// a NaN is ignored or returned), and a value the compiler must not trace back,
// so that it does not keep in registers what is cheap to compute again.
#ifndef FINETUNE_MAX3
#define FINETUNE_MAX3(out, a, b, c) asm("v_max3_f32 %0, %1, %2, %3" : "=v"(out) : "v"(a), "v"(b), "v"(c))
#define FINETUNE_OPAQUE(x) asm volatile("" : "+v"(x))
#endif

// Between a lane's LDS accesses and another lane's of the same wave: the
// hardware keeps a wave's order, and the compiler must not change it.
#ifndef FINETUNE_WAVE_FENCE
#define FINETUNE_WAVE_FENCE() __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront")
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

// Lane l's v from lane l ^ M of its wave, for M = 1, 2, or what serves in a sum
// or maximum once the lanes below M agree: the mirrored lane of its 8 (M = 4)
// or 16 (M = 8).  These move through the vector unit's data paths in a few
// cycles; the general shuffle goes through LDS (2048 x 4096 half layer norm 10.0 against 9.6 us,
// one row of 4096 2.9 against 2.6 us).
template <int M>
__device__ __forceinline__ uint32_t lane_swap(uint32_t v) {
  constexpr int kCtrl = M == 1 ? 0xB1 : M == 2 ? 0x4E : M == 4 ? 0x141 : 0x140;
  return __builtin_amdgcn_update_dpp(v, v, kCtrl, 0xf, 0xf, false);
}

// op over T consecutive lanes (T <= 64 a power of two), the result in all of
// them.  op is commutative; the order of its application is fixed.
template <int T, class F>
__device__ __forceinline__ float lanes_reduce(float v, F op) {
  auto f = [](uint32_t u) { return __builtin_bit_cast(float, u); };
  auto u = [](float x) { return __builtin_bit_cast(uint32_t, x); };
  if constexpr (T > 1) v = op(v, f(lane_swap<1>(u(v))));
  if constexpr (T > 2) v = op(v, f(lane_swap<2>(u(v))));
  if constexpr (T > 4) v = op(v, f(lane_swap<4>(u(v))));
  if constexpr (T > 8) v = op(v, f(lane_swap<8>(u(v))));
  if constexpr (T > 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(u(v), u(v), false, false);
    v = op(f(p[0]), f(p[1]));
  }
  if constexpr (T > 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(u(v), u(v), false, false);
    v = op(f(p[0]), f(p[1]));
  }
  return v;
}

// The same for the sum of a float, a double (its halves moved apart) or an int.
template <int T, class V>
__device__ __forceinline__ V lanes_sum(V v) {
  if constexpr (std::is_same_v<V, float>) {
    return lanes_reduce<T>(v, [](float a, float b) { return a + b; });
  } else if constexpr (std::is_same_v<V, int>) {
    return __builtin_bit_cast(int, lanes_reduce<T>(__builtin_bit_cast(float, v), [](float a, float b) {
      return __builtin_bit_cast(float, __builtin_bit_cast(int, a) + __builtin_bit_cast(int, b));
    }));
  } else {
    struct Halves {
      uint32_t lo, hi;
    };
    const auto moved = [](V x, auto move) {
      Halves h = __builtin_bit_cast(Halves, x);
      return __builtin_bit_cast(V, Halves{move(h.lo), move(h.hi)});
    };
    if constexpr (T > 1) v += moved(v, [](uint32_t u) { return lane_swap<1>(u); });
    if constexpr (T > 2) v += moved(v, [](uint32_t u) { return lane_swap<2>(u); });
    if constexpr (T > 4) v += moved(v, [](uint32_t u) { return lane_swap<4>(u); });
    if constexpr (T > 8) v += moved(v, [](uint32_t u) { return lane_swap<8>(u); });
    if constexpr (T > 16)
      v = moved(v, [](uint32_t u) { return __builtin_amdgcn_permlane16_swap(u, u, false, false)[0]; }) +
          moved(v, [](uint32_t u) { return __builtin_amdgcn_permlane16_swap(u, u, false, false)[1]; });
    if constexpr (T > 32)
      v = moved(v, [](uint32_t u) { return __builtin_amdgcn_permlane32_swap(u, u, false, false)[0]; }) +
          moved(v, [](uint32_t u) { return __builtin_amdgcn_permlane32_swap(u, u, false, false)[1]; });
    return v;
  }
}

// The sum over T consecutive threads of a workgroup of NT (T a power of two),
// returned to all of them.  T > 64 takes the workgroup's barrier and T / 64
// slots of `s` per group of T, which may be reused after the next barrier.
template <int T, class V>
__device__ __forceinline__ V group_sum(V v, V* s) {
  v = lanes_sum<(T < kWave ? T : kWave)>(v);
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

// Sum of v over the workgroup (NT threads, a multiple of the wave), returned
// to every thread; `s` as above.
template <int NT, class V>
__device__ __forceinline__ V block_sum(V v, V* s) {
  return group_sum<NT>(v, s);
}

// 16 bytes of elements.  STREAM: past the caches, for what is too large to be
// found there again (1 GiB read at 7.0 TB/s against 6.2, copied at 6.0 against
// 5.4 with the same loop).
template <class Io, bool STREAM = false>
__device__ __forceinline__ typename Io::Vec load_vec(const typename Io::T* p) {
  const auto* v = reinterpret_cast<const typename Io::Vec*>(p);
  if constexpr (STREAM) return __builtin_nontemporal_load(v);
  return *v;
}
template <class Io, bool STREAM = false>
__device__ __forceinline__ void store_vec(typename Io::T* p, typename Io::Vec v) {
  auto* q = reinterpret_cast<typename Io::Vec*>(p);
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

// The columns [begin, end) of a row (rows start at any element): 16-byte pieces
// from the first 128-byte line on, up to `last`, and the columns before and
// after them.  Pieces at odd addresses straddle lines: reading 5808 rows of
// 50001 bf16 took 170 us from the row's start, 148 us from the first address
// divisible by 16, and 141 us from the first line on (their gradient: 281, 260,
// 248 us).
template <class Io, int LINE = 128>
struct Pieces {
  int begin, first, last, end;
  __device__ __forceinline__ Pieces(const typename Io::T* row, int b, int e) : begin(b), end(e) {
    constexpr int S = sizeof(typename Io::T), L = LINE / S;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row + b) / S % L);
    first = b + (L - off) % L;
    if (first > e) first = e;
    last = first + (e - first) / Io::kVec * Io::kVec;
  }
  // f(column) for the columns outside the pieces
  template <int NT, class F>
  __device__ __forceinline__ void rest(F f) const {
    const int head = first - begin, n = head + end - last;
    for (int t = threadIdx.x; t < n; t += NT) f(t < head ? begin + t : last + t - head);
  }
};

}  // namespace finetune
