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
constexpr int kClipBytes = 16384;   // of a chunk, the unit of work: four 16-byte pieces a thread
constexpr int kClipPieces = kClipBytes / 16 / kClipThreads;
constexpr int kClipGroups = 2048;   // workgroups of a launch at most: 8 a compute unit, and one partial sum each
constexpr uint32_t kClipEntry = 1u << 30;  // elements of a table's entry stay below this
constexpr int kClipLine = 128;      // chunks start at addresses divisible by this

// The tensors of one launch: the table travels in the kernel's arguments, as
// many as fit 4 KB with them.  APART: out is elsewhere.  An entry's elements
// (below 2^30) and its type share a word: with 8 bytes for the count and a byte
// for the type a table held 128, and 288 tensors, three launches a pass, took
// 38 us, 30 us with these.
template <int MOST, bool APART>
struct ClipTable {
  static constexpr int kMost = MOST;
  static constexpr bool kApart = APART;
  const void* in[MOST];
  void* to[APART ? MOST : 1];
  uint32_t count[MOST];  // type * 2^30 + elements
  int first[MOST + 1];   // first chunk of each tensor within the launch
  int n;
  __host__ __device__ void* out(int i) const { return APART ? to[APART ? i : 0] : const_cast<void*>(in[i]); }
};
using ClipHere = ClipTable<232, false>;
using ClipApart = ClipTable<156, true>;
static_assert(sizeof(ClipHere) <= 3800 && sizeof(ClipApart) <= 3800, "kernel arguments are limited to 4 KB");

// Elements between the last 128-byte line before p and p: chunk k of a tensor
// holds its elements [k N - lead, (k + 1) N - lead), N = 16 KB of them, so that
// every chunk but the first starts on a line.
__host__ __device__ inline int clip_lead(const void* p, int size) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) % kClipLine) / size;
}

// The tensor that chunk c belongs to, at or after tensor i: the last whose
// first chunk is <= c.
template <class Table>
__device__ __forceinline__ int tensor_of(const Table& t, int c, int i) {
  if (c < t.first[i + 1]) return i;
  int lo = i + 1, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// f(storage type, tensor's pointer in, out, begin, end) for every chunk of this
// workgroup, dealt out in turn so that all workgroups read one region at a
// time.  BACK: a tensor's last chunk first.  `at` of a tensor is the pointer
// whose lines the chunks follow.
template <bool BACK, class Table, class F>
__device__ __forceinline__ void for_chunks(const Table& t, F f) {
  const int chunks = t.first[t.n];
  int i = 0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    i = tensor_of(t, c, i);
    const auto with = [&](auto io) {
      using T = typename decltype(io)::T;
      constexpr int N = kClipBytes / sizeof(T);
      const int64_t k = BACK ? t.first[i + 1] - 1 - c : c - t.first[i];
      const void* lines = BACK ? t.out(i) : t.in[i];
      const int64_t a = k * N - clip_lead(lines, sizeof(T)), b = a + N, n = t.count[i] & (kClipEntry - 1);
      f(io, static_cast<const T*>(t.in[i]), static_cast<T*>(t.out(i)), a > 0 ? a : 0, b < n ? b : n, a, c);
    };
    const int type = t.count[i] / kClipEntry;
    if (type == 0)
      with(F32{});
    else if (type == 1)
      with(Bf16{});
    else
      with(F16{});
  }
}

// A chunk [begin, end) of a tensor whose lines start at `origin` (at or before
// begin): piece(slot, column) for the thread's whole 16-byte pieces, then
// one(column) for the columns that a cut first or last piece leaves.
template <class Io, class Piece, class One>
__device__ __forceinline__ void for_pieces(int64_t origin, int64_t begin, int64_t end, Piece piece, One one) {
  constexpr int V = Io::kVec;
  const int head = static_cast<int>(begin - origin) % V;  // columns missing from the first piece
  const int64_t first = begin + (head ? V - head : 0), last = first < end ? first + (end - first) / V * V : first;
#pragma unroll
  for (int u = 0; u < kClipPieces; ++u) {
    const int64_t j = origin + (u * kClipThreads + static_cast<int>(threadIdx.x)) * V;
    if (j >= first && j < last) piece(u, j);
  }
  const int t = threadIdx.x, before = static_cast<int>((first < end ? first : end) - begin);
  if (t < before)
    one(begin + t);
  else if (last + t - before < end && last >= first && first < end)
    one(last + t - before);
}

// partial[workgroup] = the sum of squares of its chunks; those below `keep` are
// read past the caches
__global__ void __launch_bounds__(kClipThreads) grad_square_kernel(ClipHere t, int keep, double* partial) {
  __shared__ double s[kClipThreads / kWave];
  double sum[2] = {0.0, 0.0};
  for_chunks<false>(
      t, [&](auto io, const auto* g, auto*, int64_t begin, int64_t end, int64_t origin, int c) {
        using Io = decltype(io);
        constexpr int V = Io::kVec;
        typename Io::Vec raw[kClipPieces] = {};  // pieces that are not there add zero
        typename Io::T single = 0;
        const auto load = [&](auto stream) {
          for_pieces<Io>(
              origin, begin, end, [&](int u, int64_t j) { raw[u] = load_vec<Io, decltype(stream)::value>(g + j); },
              [&](int64_t j) { single = g[j]; });
        };
        if (c < keep)
          load(std::true_type{});
        else
          load(std::false_type{});
        const auto add = [&](auto v, int k) {
          const double x = Io::widen(v);
          sum[k % 2] = __builtin_fma(x, x, sum[k % 2]);
        };
#pragma unroll
        for (int k = 0; k < kClipPieces * V; ++k) add(raw[k / V][k % V], k);
        add(single, 0);
      });
  const double all = block_sum<kClipThreads>(sum[0] + sum[1], s);
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
// kernel that does.  The tables come in reverse and so do a tensor's chunks:
// what the squares read last is still in the 256 MB cache.
template <class Table, bool STREAM>
__global__ void __launch_bounds__(kClipThreads)
    grad_scale_kernel(Table t, const double* partial, int64_t parts, double max_norm, double eps, float* norm) {
  __shared__ double s[kClipThreads / kWave];
  const double a = norm_of(partial, parts, s);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = static_cast<float>(a);
  const double q = max_norm / (a + eps);
  const float f = q > 1.0 ? 1.0f : static_cast<float>(q);
  for_chunks<true>(
      t, [&](auto io, const auto* g, auto* o, int64_t begin, int64_t end, int64_t origin, int) {
        using Io = decltype(io);
        constexpr int V = Io::kVec;
        if (f == 1.0f && g == o) return;  // nothing to change in place
        typename Io::Vec raw[kClipPieces];
        for_pieces<Io>(
            origin, begin, end, [&](int u, int64_t j) { raw[u] = load_vec<Io, STREAM>(g + j); }, [](int64_t) {});
        for_pieces<Io>(
            origin, begin, end,
            [&](int u, int64_t j) {
#pragma unroll
              for (int k = 0; k < V; ++k) raw[u][k] = Io::narrow(Io::widen(raw[u][k]) * f);
              store_vec<Io, STREAM>(o + j, raw[u]);
            },
            [&](int64_t j) { o[j] = Io::narrow(Io::widen(g[j]) * f); });
      });
}

}  // namespace finetune
