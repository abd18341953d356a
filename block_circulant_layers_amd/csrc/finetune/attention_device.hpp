// attention_device.hpp -- what the attention kernels share: matrix products of
// 32 x 32 blocks, tiles in LDS, the grid, masks and the position bias.
//
// A product D += A B of a 32 x 16 and a 16 x 32 block takes one matrix
// instruction for 16-bit types and eight for fp32.  Lane l holds of A the row
// l % 32 and of B the column l % 32, each the eight elements 8 (l / 32) .. + 7 of
// the sum's index, and of D the column l % 32 and the sixteen rows
// 8 (r / 4) + 4 (l / 32) + r % 4.  The order of the sum's index is free as long
// as A and B share it.  So a block of D, rounded, is a B operand of the next
// product as it lies: registers 0..7 are the eight rows {4g .. 4g + 3,
// 8 + 4g .. 8 + 4g + 3} (g = l / 32) of its first 16 rows, registers 8..15 those
// of the second; the A operand then takes its columns in that order.  Scores
// never pass through LDS.
#pragma once

#include "device.hpp"
#include "relative_bias.hpp"

namespace finetune {

typedef float Acc __attribute__((ext_vector_type(16)));
typedef short ShortFour __attribute__((ext_vector_type(4)));

// Four 16-bit elements by the LDS's transposed read: 16 lanes give the addresses of 4 elements each, together 4 rows
// of 16 (lanes 4 r .. 4 r + 3 row r), and lane i gets the i-th element of each row.  A host build defines it otherwise.
#ifndef FINETUNE_READ_TRANSPOSED
#define FINETUNE_READ_TRANSPOSED(p) \
  __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) finetune::ShortFour*)(p))
#endif

template <class Io>
struct Mma;
template <>
struct Mma<Bf16> {
  typedef __bf16 Frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ Acc mul(Frag a, Frag b, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ __bf16 narrow(float v) { return static_cast<__bf16>(v); }
};
template <>
struct Mma<F16> {
  typedef _Float16 Frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ Acc mul(Frag a, Frag b, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ _Float16 narrow(float v) { return static_cast<_Float16>(v); }
};
template <>
struct Mma<F32> {
  typedef float Frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ Acc mul(Frag a, Frag b, Acc c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ float narrow(float v) { return v; }
};

// eight registers of a block of D from `at` on as a B operand
template <class Io>
__device__ __forceinline__ typename Mma<Io>::Frag frag_of(const Acc& a, int at) {
  typename Mma<Io>::Frag f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = Mma<Io>::narrow(a[at + j]);
  return f;
}

__device__ __forceinline__ Acc zero_acc() {
  Acc a;
#pragma unroll
  for (int r = 0; r < 16; ++r) a[r] = 0.0f;
  return a;
}

// v of the other half of the wave joined with this lane's by op
template <class F>
__device__ __forceinline__ float halves(float v, F op) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t low = p[0], high = p[1];  // (a cast of p[1] itself would be compiled as one of p[0])
  return op(__builtin_bit_cast(float, low), __builtin_bit_cast(float, high));
}
__device__ __forceinline__ float halves_sum(float v) {
  return halves(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float halves_max(float v) {
  return halves(v, [](float a, float b) { return fmaxf(a, b); });
}

// 2^x, and 2^(x + kLift): half's smallest normal number is 2^-14, so its probabilities are held 2^8 times as
// large (exact, and taken back in the sums that they enter); the other types have the exponents of fp32.
template <class Io>
constexpr float kLift = std::is_same_v<Io, F16> ? 8.0f : 0.0f;
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// ---------------------------------------------------------------------------
// tiles in LDS: rows of DP elements, a power of two apart, in pieces of 16
// bytes whose order is permuted from row to row.  Two ways of reading must not
// meet in the banks: 32 lanes take one piece of 32 rows (A operands along a
// row: the permutation differs between 8 neighbouring rows), and 16 lanes take
// 32 bytes each of 4 neighbouring rows (transposed reads: it differs by pairs
// of pieces there).
// ---------------------------------------------------------------------------
template <class Io, int DP>
struct Tile {
  using T = typename Io::T;
  typedef T Piece __attribute__((ext_vector_type(Io::kVec)));
  static constexpr int V = Io::kVec;
  static constexpr int kStride = DP <= 32 ? 32 : DP <= 64 ? 64 : 128;
  static constexpr int kPieces = DP / V;                       // of a row that hold data
  static constexpr int kLine = kStride * int(sizeof(T)) / 16;  // pieces from row to row
  static constexpr int bytes(int rows) { return rows * kStride * int(sizeof(T)); }

  static __device__ __forceinline__ int turn(int row) {
    if constexpr (kLine < 8) return (row >> 1) & 3;
    return ((row & 3) << 1) | ((row >> 2) & 1);
  }
  static __device__ __forceinline__ int at(int row, int piece) { return row * kStride + ((piece ^ turn(row)) * V); }

  // A operand for lane l: rows r0 + l % 32, elements 16 c + 8 (l / 32) .. + 7
  static __device__ __forceinline__ typename Mma<Io>::Frag rows(const T* s, int r0, int c, int l) {
    const int row = r0 + l % 32, g = l / 32;
    typename Mma<Io>::Frag f;
    if constexpr (V == 8) {
      f = __builtin_bit_cast(typename Mma<Io>::Frag, *reinterpret_cast<const Piece*>(s + at(row, 2 * c + g)));
    } else {
      const Piece lo = *reinterpret_cast<const Piece*>(s + at(row, 4 * c + 2 * g)),
                  hi = *reinterpret_cast<const Piece*>(s + at(row, 4 * c + 2 * g + 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = lo[j], f[4 + j] = hi[j];
    }
    return f;
  }

  // A operand of the transposed tile: its row l % 32 is column c0 + l % 32 here, its columns are the rows
  // r0 + {4g .. 4g + 3, 8 + 4g .. 8 + 4g + 3}.
  static __device__ __forceinline__ typename Mma<Io>::Frag cols(const T* s, int r0, int c0, int l) {
    const int g = l / 32;
    typename Mma<Io>::Frag f;
    if constexpr (V == 8) {
      const int col = c0 + 16 * (l % 32 / 16) + 4 * (l % 4), row = r0 + 4 * g + l % 16 / 4;
      struct {
        ShortFour a, b;
      } both;
      both.a = FINETUNE_READ_TRANSPOSED(s + at(row, col / 8) + col % 8);
      both.b = FINETUNE_READ_TRANSPOSED(s + at(row + 8, col / 8) + col % 8);
      f = __builtin_bit_cast(typename Mma<Io>::Frag, both);
    } else {
      const int col = c0 + l % 32;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = s[at(r0 + 8 * (j / 4) + 4 * g + j % 4, col / 4) + col % 4];
    }
    return f;
  }
};

// The 16 bytes of elements c .. of a row of d elements, zeros from d on.  Where rows end inside a piece the last one is
// loaded from the row's last 16 bytes and shifted into place, so that nothing past the row is read.
template <class Io>
__device__ __forceinline__ auto piece_of(const typename Io::T* row, int c, int d) {
  using T = typename Io::T;
  constexpr int V = Io::kVec;
  typedef T Piece __attribute__((ext_vector_type(V)));
  typedef unsigned __int128 Bits;
  const auto load = [](const T* p) { return __builtin_bit_cast(Piece, *reinterpret_cast<const typename Io::Vec*>(p)); };
  Piece v = {};
  if (d % V == 0) {
    v = load(row + (c < d ? c : 0));
  } else if (d > V) {
    const int start = c < d - V ? c : d - V, skip = c - start;
    v = load(row + start);
    v = __builtin_bit_cast(Piece, __builtin_bit_cast(Bits, v) >> ((skip & (V - 1)) * 8 * int(sizeof(T))));
  } else {
#pragma unroll
    for (int x = 0; x < V; ++x)
      if (c + x < d) v[x] = row[c + x];
  }
  return c < d ? v : Piece{};
}

// use(i, load(i)) for i = 0 .. N - 1, the operands fetched from LDS a group of G ahead (0: as the compiler likes): an operand takes its product
// 32 cycles and LDS some 200, and the compiler by itself fetches one ahead.
template <class Io, int N, int G, class L, class U>
__device__ __forceinline__ void fetched_ahead(L load, U use) {
  static_assert(G == 0 || N % G == 0, "whole groups");
  if constexpr (G == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) use(i, load(i));
  }
  typename Mma<Io>::Frag f[2][G > 0 ? G : 1];
#pragma unroll
  for (int i = 0; i < G; ++i) f[0][i] = load(i);
#pragma unroll
  for (int s = 0; s < (G > 0 ? N / G : 0); ++s) {
    if ((s + 1) * G < N) {
#pragma unroll
      for (int i = 0; i < G; ++i) f[(s + 1) % 2][i] = load((s + 1) * G + i);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < G; ++i) use(s * G + i, f[s % 2][i]);
  }
}
// how many operands ahead, of N: four of the 16-bit types (dk and dv of the long case in attention_bwd.hpp 1240 us
// without, 1040 with; the forward the same either way)
template <class Io, int N>
constexpr int kAheadOf = sizeof(typename Io::T) == 4 ? 0 : N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 0;

// A lane's number that the compiler must not trace back: what is worked out from it takes no registers meanwhile.
__device__ __forceinline__ int opaque(int l) {
  FINETUNE_OPAQUE(l);
  return l;
}

// A thread's share of a tile of ROWS rows on its way from global memory to LDS,
// held in registers in between so that the loads run under the tile before.
// Rows outside [lo, hi) and elements from d on become zeros and are not read.
template <class Io, int DP, int ROWS, int NT>
struct Stage {
  using T = typename Io::T;
  using L = Tile<Io, DP>;
  static constexpr int N = ROWS * L::kPieces / NT;
  static_assert(N * NT == ROWS * L::kPieces, "whole pieces for each thread");
  typename L::Piece r[N];
  uint32_t zeros;  // bit n: the n-th piece is to be zeros; applied on the way to LDS, so that no load is waited for here

  // of thread t's n-th piece
  static __device__ __forceinline__ int row(int t, int n) { return (t + n * NT) / L::kPieces; }
  static __device__ __forceinline__ int piece(int t, int n) { return (t + n * NT) % L::kPieces; }

  __device__ __forceinline__ void load(const T* base, int64_t stride, int64_t row0, int64_t lo, int64_t hi, int d) {
    const int t = opaque(threadIdx.x);
    zeros = 0;
    // A tile of whole rows of whole pieces is read without a test, with 32-bit offsets from its first row.
    if (row0 >= lo && row0 + ROWS <= hi && d % L::V == 0 && stride < (int64_t(1) << 24)) {
      const T* first = base + row0 * stride;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = piece(t, n) * L::V;
        const uint32_t at = row(t, n) * static_cast<uint32_t>(stride) + (c < d ? c : 0);
        r[n] = __builtin_bit_cast(typename L::Piece, *reinterpret_cast<const typename Io::Vec*>(first + at));
        zeros |= c < d ? 0 : 1u << n;
      }
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int64_t j = row0 + row(t, n), near = j < lo ? lo : j >= hi ? hi - 1 : j;
        r[n] = piece_of<Io>(base + near * stride, piece(t, n) * L::V, d);
        zeros |= near == j ? 0 : 1u << n;
      }
    }
  }
  __device__ __forceinline__ void store(T* s) {
    const int t = opaque(threadIdx.x);
    if (__any(zeros != 0)) {
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (zeros >> n & 1) r[n] = typename L::Piece{};
    }
#pragma unroll
    for (int n = 0; n < N; ++n) *reinterpret_cast<typename L::Piece*>(s + L::at(row(t, n), piece(t, n))) = r[n];
  }
};

// B operand straight from a row in global memory: elements 16 c + 8 g .. + 7, zeros from d on
template <class Io>
__device__ __forceinline__ typename Mma<Io>::Frag row_frag(const typename Io::T* row, bool valid, int c, int d) {
  const int x0 = 16 * c + 8 * (threadIdx.x % kWave / 32);
  typename Mma<Io>::Frag f;
  if constexpr (Io::kVec == 8) {
    const auto v = piece_of<Io>(row, x0, d);
    f = __builtin_bit_cast(typename Mma<Io>::Frag, valid ? v : decltype(v){});
  } else {
    const auto lo = piece_of<Io>(row, x0, d), hi = piece_of<Io>(row, x0 + 4, d);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = valid ? lo[j] : 0.0f, f[4 + j] = valid ? hi[j] : 0.0f;
  }
  return f;
}

// Four values of a block of D, consecutive elements x0 .. x0 + 3 of a row, rounded and stored up to d
template <class Io>
__device__ __forceinline__ void store_four(typename Io::T* row, int x0, int d, float a, float b, float c, float e) {
  using T = typename Io::T;
  typedef T Four __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  const Four v = {Io::narrow(a), Io::narrow(b), Io::narrow(c), Io::narrow(e)};
  if (x0 + 4 <= d) {
    *reinterpret_cast<Four*>(row + x0) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (x0 + i < d) row[x0 + i] = v[i];
  }
}

// ---------------------------------------------------------------------------
// shapes, grid, masks
// ---------------------------------------------------------------------------
struct View {  // element (b, t, h, x) at p[b * sb + t * st + h * sh + x]
  void* p;
  int64_t sb, st, sh;
  template <class T>
  __device__ __forceinline__ T* at(int64_t b, int64_t t, int64_t h) const {
    return static_cast<T*>(p) + b * sb + t * st + h * sh;
  }
};

struct Problem {
  int batch, tq, tk, heads, kv_heads, d, group, causal;
  float scale, scale2;  // scale, and scale * log2(e)
  const int32_t *begin, *end;
  const float* table;
};

// the keys [lo, hi) that count for sequence b
__device__ __forceinline__ void span_of(const Problem& a, int b, int& lo, int& hi) {
  lo = a.begin ? a.begin[b] : 0;
  hi = a.end ? a.end[b] : a.tk;
  lo = lo < 0 ? 0 : lo > a.tk ? a.tk : lo;
  hi = hi < lo ? lo : hi > a.tk ? a.tk : hi;
}

// Which work a workgroup takes: `per` consecutive items of each of `units`
// (sequence, head group).  Workgroups go around the 8 XCDs in turn, so where the
// units divide evenly each XCD gets whole units, whose keys and values then
// come from its own L2.
__device__ __forceinline__ void locate(uint32_t block, uint32_t units, uint32_t per, uint32_t& unit, uint32_t& item) {
  if (units % 8 == 0) {
    const uint32_t n = block / 8;
    unit = n / per * 8 + block % 8;
    item = n % per;
  } else {
    unit = block / per;
    item = block % per;
  }
}

// The bias of one head by relative position, times log2(e), in LDS: positions -reach - kEdge .. reach + kEdge, so
// that a block of 32 x 32 scores that holds any position inside [-reach, reach] reads no further.
constexpr int kEdge = 63;
// a wave's scratch for one block of scores in fp32, its rows an odd number of banks apart, and 32 floats before and
// after them, where reads along a diagonal begin and end
constexpr int kBlockLine = 33, kBlockFloats = 64 + 32 * kBlockLine;
__host__ __device__ __forceinline__ int bias_line(const Buckets& b) { return 2 * (b.reach + kEdge) + 1; }
template <int NT>
__device__ __forceinline__ void load_bias(float* line, const float* table, int heads, int h, const Buckets& b) {
  const int n = bias_line(b);
  for (int t = threadIdx.x; t < n; t += NT) line[t] = table[int64_t(b.of(t - b.reach - kEdge)) * heads + h] * kLog2e;
}

}  // namespace finetune
