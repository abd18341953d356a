// attention_fwd.hpp -- attention in one pass over the keys, with the running maximum and sum of the softmax.
//
// A workgroup of four waves takes 128 rows, 32 a wave, and walks over the keys
// 64 at a time; keys and values come through LDS, the rows of q stay in
// registers.  Scores are computed transposed (keys x rows), so that a lane has
// all its scores of one row: the maximum and the sum need one exchange between
// the two halves of the wave, and the probabilities are the operand of the
// product with the values as they lie (attention_device.hpp).  They are rounded
// to the storage type there; their sum is not.
//
// Two waves a SIMD take turns at LDS, matrix and vector units.  2 x 4096 tokens,
// 32 heads over 8 of 128, bf16: 715 us, 769 TFLOP/s (a library product of 8192^3
// 1200); 2 x 4096, 32 heads of 64: 395 us, 690 TFLOP/s, bound by the softmax's
// vector instructions.  4 x 512 causal fp16 is one round of 2 to 8 tiles a
// workgroup: 29 us for 67 MB.
#pragma once

#include "attention_device.hpp"

namespace finetune {

constexpr int kAttnThreads = 256, kAttnRows = 128, kAttnKeys = 64;

// waves a SIMD that the registers of a kernel are cut for: fp32 operands of 128 elements take twice the registers
template <class Io, int DP, bool BIAS>
constexpr int kFwdWaves = DP > 64 && (sizeof(typename Io::T) == 4 || (BIAS && DP > 96)) ? 1 : 2;

// Where the keys are split over workgroups (few rows): each leaves its
// unnormalised sums, maximum (in units of log2) and sum of exponentials.
struct FwdParts {
  float* o;      // [splits, rows, d]
  float* stats;  // [splits, rows, 2]
  int splits;
};

// Rows are (query, head) pairs: with `pack` heads of a group side by side, row r of a head group is query r / pack,
// head r % pack.  pack is 1 or the group's size.
template <class Io, int DP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads, (kFwdWaves<Io, DP, BIAS>)) void attention_fwd_kernel(Problem a, View q, View k, View v, View o,
                                                                        float* lse, FwdParts parts, int pack,
                                                                        Buckets buckets) {
  using T = typename Io::T;
  using M = Mma<Io>;
  using L = Tile<Io, DP>;
  constexpr int DC = DP / 16, DB = DP / 32, KB = kAttnKeys / 32;
  FINETUNE_DYNAMIC_LDS(attention_lds);
  T* sk = reinterpret_cast<T*>(attention_lds);
  T* sv = sk + L::bytes(kAttnKeys) / sizeof(T);
  float* line = reinterpret_cast<float*>(sv + L::bytes(kAttnKeys) / sizeof(T));

  const int rows = a.tq * pack, tiles = (rows + kAttnRows - 1) / kAttnRows;
  uint32_t unit, item;
  locate(blockIdx.x, a.batch * a.kv_heads, a.group / pack * tiles * parts.splits, unit, item);
  const int b = static_cast<int>(unit / a.kv_heads), kvh = static_cast<int>(unit % a.kv_heads);
  const int split = static_cast<int>(item % parts.splits);
  item /= parts.splits;
  const int tile = tiles - 1 - static_cast<int>(item % tiles);  // a causal mask leaves the last tiles the most keys
  const int h0 = kvh * a.group + static_cast<int>(item / tiles) * pack;

  const int l = threadIdx.x % kWave, wave = threadIdx.x / kWave, g = l / 32;
  const int w0 = tile * kAttnRows + wave * 32, row = w0 + l % 32;
  const bool live = row < rows;
  const int i = row / pack, h = h0 + row % pack;
  const int off = a.tk - a.tq;

  int lo, hi;
  span_of(a, b, lo, hi);
  const int hi_row = a.causal && i + off + 1 < hi ? i + off + 1 : hi;  // this row's keys are [lo, hi_row)
  const int first_i = w0 / pack;                                       // of the wave's rows
  const int wave_hi = a.causal && first_i + off + 1 < hi ? first_i + off + 1 : hi;  // what all its rows see ends here
  const int wave_i = (w0 + 31) / pack;
  const int wave_end = a.causal && wave_i + off + 1 < hi ? wave_i + off + 1 : hi;  // what any of its rows sees
  int last_i = (tile * kAttnRows + kAttnRows - 1) / pack;
  if (last_i > a.tq - 1) last_i = a.tq - 1;
  int tile_hi = a.causal && last_i + off + 1 < hi ? last_i + off + 1 : hi;  // what any row of the tile sees
  int k0 = lo / kAttnKeys, k1 = tile_hi > lo ? (tile_hi + kAttnKeys - 1) / kAttnKeys : k0;
  if (parts.splits > 1) {
    const int per = (k1 - k0 + parts.splits - 1) / parts.splits;
    k0 += split * per;
    k1 = k0 + per < k1 ? k0 + per : k1;
  }

  typename M::Frag qf[DC];
  const T* qrow = q.at<const T>(b, live ? i : 0, live ? h : h0);
#pragma unroll
  for (int c = 0; c < DC; ++c) qf[c] = row_frag<Io>(qrow, live, c, a.d);

  if constexpr (BIAS) load_bias<kAttnThreads>(line, a.table, a.heads, h0, buckets);

  Acc acc[DB];
#pragma unroll
  for (int n = 0; n < DB; ++n) acc[n] = zero_acc();
  float top = -INFINITY, total = 0.0f;  // the running maximum (log2 units) and this half's sum

  const T* kbase = k.at<const T>(b, 0, kvh);
  const T* vbase = v.at<const T>(b, 0, kvh);
  Stage<Io, DP, kAttnKeys, kAttnThreads> nk, nv;
  if (k0 < k1) {
    nk.load(kbase, k.st, int64_t(k0) * kAttnKeys, lo, hi, a.d);
    nv.load(vbase, v.st, int64_t(k0) * kAttnKeys, lo, hi, a.d);
  }
  for (int t = k0; t < k1; ++t) {
    __syncthreads();
    nk.store(sk);
    nv.store(sv);
    __syncthreads();
    if (t + 1 < k1) {
      nk.load(kbase, k.st, int64_t(t + 1) * kAttnKeys, lo, hi, a.d);
      nv.load(vbase, v.st, int64_t(t + 1) * kAttnKeys, lo, hi, a.d);
    }
    const int j0 = t * kAttnKeys;
    if (j0 >= wave_end) continue;  // none of the wave's rows sees these keys
    Acc x[KB];
#pragma unroll
    for (int n = 0; n < KB; ++n) x[n] = zero_acc();
    fetched_ahead<Io, KB * DC, kAheadOf<Io, KB * DC>>(
        [&](int m) { return L::rows(sk, 32 * (m % KB), m / KB, l); },
        [&](int m, auto f) { x[m % KB] = M::mul(f, qf[m / KB], x[m % KB]); });
    if constexpr (BIAS) {
#pragma unroll
      for (int n = 0; n < KB; ++n) {
        const int j = j0 + 32 * n;
        const int rel_lo = j - (w0 + 31) - off, rel_hi = j + 31 - w0 - off;  // of the block (pack is 1)
        if (rel_hi <= -buckets.reach || rel_lo >= buckets.reach) {
          const float one = line[rel_lo >= buckets.reach ? 2 * (buckets.reach + kEdge) : 0];
#pragma unroll
          for (int r = 0; r < 16; ++r) x[n][r] = fmaf(x[n][r], a.scale2, one);
        } else {
          const float* from = line + (j + 4 * g - row - off + buckets.reach + kEdge);
#pragma unroll
          for (int r = 0; r < 16; ++r) x[n][r] = fmaf(x[n][r], a.scale2, from[8 * (r / 4) + r % 4]);
        }
      }
    }
    if (j0 < lo || j0 + kAttnKeys > wave_hi) {
#pragma unroll
      for (int n = 0; n < KB; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = j0 + 32 * n + 8 * (r / 4) + 4 * g + r % 4;
          if (j < lo || j >= hi_row) x[n][r] = -INFINITY;
        }
    }
    const float unit2 = BIAS ? 1.0f : a.scale2;
    float m = x[0][0];
#pragma unroll
    for (int n = 0; n < KB; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) m = fmaxf(m, x[n][r]);
    m = fmaxf(top, halves_max(m) * unit2);
    const float base = m == -INFINITY ? 0.0f : m;
    const float keep = exp2_of(top - base);
    const float shift = kLift<Io> - base;
    float s = 0.0f;
#pragma unroll
    for (int n = 0; n < KB; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        x[n][r] = exp2_of(fmaf(x[n][r], unit2, shift));
        s += x[n][r];
      }
    total = total * keep + s;
    if (__any(m > top)) {  // rows whose maximum stays keep their sums as they are
#pragma unroll
      for (int n = 0; n < DB; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[n][r] *= keep;
    }
    top = m;
    typename M::Frag p[2 * KB];
#pragma unroll
    for (int c = 0; c < 2 * KB; ++c) p[c] = frag_of<Io>(x[c / 2], 8 * (c % 2));
    fetched_ahead<Io, 2 * KB * DB, kAheadOf<Io, 2 * KB * DB>>(
        [&](int m) { return L::cols(sv, 16 * (m / DB), 32 * (m % DB), l); },
        [&](int m, auto f) { acc[m % DB] = M::mul(f, p[m / DB], acc[m % DB]); });
  }
  total = halves_sum(total);
  if (!live) return;
  const int64_t at = (int64_t(b) * a.heads + h) * a.tq + i;
  if (parts.splits > 1) {
    const int64_t place = split * (int64_t(a.batch) * a.heads * a.tq) + at;
    float* out = parts.o + place * a.d;
#pragma unroll
    for (int n = 0; n < DB; ++n)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        store_four<F32>(out, 32 * n + 2 * r + 4 * g, a.d, acc[n][r], acc[n][r + 1], acc[n][r + 2], acc[n][r + 3]);
    if (g == 0) {
      parts.stats[place * 2] = top;
      parts.stats[place * 2 + 1] = total;
    }
    return;
  }
  const float inv = 1.0f / total;
  const auto value = [&](float x) { return total == 0.0f ? 0.0f : x * inv; };  // (0 also beside values of infinity)
  T* out = o.at<T>(b, i, h);
#pragma unroll
  for (int n = 0; n < DB; ++n)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      store_four<Io>(out, 32 * n + 2 * r + 4 * g, a.d, value(acc[n][r]), value(acc[n][r + 1]), value(acc[n][r + 2]),
                     value(acc[n][r + 3]));
  if (g == 0) lse[at] = total == 0.0f ? -INFINITY : (top - kLift<Io> + log2f(total)) * kLn2;
}

// The parts of a row joined: their weights first, one a lane, then the columns, two a lane, by LANES waves that
// each sum every LANES-th part: eight waves for more than eight parts (32 rows of 32 parts 7.5 us, 29 with one wave that
// reads a part after another), one for fewer (20000 rows of two parts 11 us, 37 with eight).
constexpr int kMaxSplits = kWave;
template <class Io, int LANES>
__global__ __launch_bounds__(kWave* LANES) void attention_join_kernel(Problem a, View o, float* lse, FwdParts parts) {
  using T = typename Io::T;
  __shared__ float weight[kMaxSplits], sums[LANES][2][kWave];
  const int64_t at = blockIdx.x, all = int64_t(a.batch) * a.heads * a.tq;
  const int l = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const float* stat = parts.stats + (l < parts.splits ? l * all + at : at) * 2;
  const float own = l < parts.splits ? stat[0] : -INFINITY;
  const float top = lanes_reduce<kWave>(own, [](float x, float y) { return fmaxf(x, y); });
  const float scale = exp2_of(own - (top == -INFINITY ? 0.0f : top));
  const float total = lanes_sum<kWave>(l < parts.splits ? stat[1] * scale : 0.0f);
  if (wave == 0) weight[l] = scale;
  __syncthreads();
  float x = 0.0f, y = 0.0f;
  const float* from = parts.o + at * a.d;
  const int64_t step = all * a.d;
#pragma unroll 8
  for (int s = wave; s < parts.splits; s += LANES) {
    const float* p = from + s * step;
    if (l < a.d) x = fmaf(p[l], weight[s], x);
    if (l + kWave < a.d) y = fmaf(p[l + kWave], weight[s], y);
  }
  if constexpr (LANES > 1) {
    sums[wave][0][l] = x;
    sums[wave][1][l] = y;
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int n = 1; n < LANES; ++n) x += sums[n][0][l], y += sums[n][1][l];
  }
  const int i = static_cast<int>(at % a.tq);
  const int64_t bh = at / a.tq;
  T* out = o.at<T>(bh / a.heads, i, bh % a.heads);
  const float inv = 1.0f / total;
  if (l < a.d) out[l] = Io::narrow(total == 0.0f ? 0.0f : x * inv);
  if (l + kWave < a.d) out[l + kWave] = Io::narrow(total == 0.0f ? 0.0f : y * inv);
  if (threadIdx.x == 0) lse[at] = total == 0.0f ? -INFINITY : (top - kLift<Io> + log2f(total)) * kLn2;
}

}  // namespace finetune
