// attention_bwd.hpp -- the attention's gradients from q, k, v, o, lse and dout; the probabilities are computed again.
//
// Two kernels, each of which owns what it sums, so that no sum goes through
// atomics in memory and results repeat bit for bit:
//   dq: a workgroup owns 128 queries and walks over the keys,
//   dk and dv: a workgroup owns 128 keys of a key head and walks over the
//   queries of every head that shares it.
// Both compute scores and dp, so seven products in place of the five that the
// gradients need; one kernel with dq summed by atomics would save two and lose
// the fixed order.  The first one also forms delta, which the second reads.
//
// Bound by LDS latency at two waves a SIMD (dq) or one (dk and dv of more than 64
// elements, whose sums, keys and values take 192 registers): 2 x 4096 causal
// tokens, 32 heads over 8 of 128, bf16 670 and 950 us, 430 TFLOP/s of the five
// products together; 2 x 4096, 32 heads of 64 1340 us, 510 TFLOP/s.
#pragma once

#include <limits.h>

#include "attention_fwd.hpp"

namespace finetune {

// fp32 operands of 128 elements: the kernel of dk and dv takes 32 queries at a time in place of 64, and loads them
// only when it needs them, to do without registers in memory.
template <class Io, int DP>
constexpr bool kBwdTight = sizeof(typename Io::T) == 4 && DP > 64;
template <class Io, int DP>
constexpr int kBwdQueries = kBwdTight<Io, DP> ? 32 : 64;
// floats in LDS of such a step: the tiles of q and dout, and for each query kLift - lse in log2 units, -delta, peak
template <class Io, int DP>
constexpr int kTileSet = 2 * Tile<Io, DP>::bytes(kBwdQueries<Io, DP>) / 4 + 3 * kBwdQueries<Io, DP>;

// Waves a SIMD that the registers are cut for.  On the long case above dq took 830 us at one wave and 530 at two (before
// ds had two parts); dk and dv 1040 us at one, where two keep registers in memory or the values in LDS (1104 us).
template <class Io, int DP, bool BIAS>
constexpr int kDqWaves = (sizeof(typename Io::T) == 4 && DP > 32) || (BIAS && DP > 96) ? 1 : 2;
// operands fetched ahead by the kernel of dq, of N: four at 128 elements keep registers in memory (590 us against 530)
template <class Io, int DP, int N>
constexpr int kDqGroup = DP > 96 ? 0 : kAheadOf<Io, N>;
template <class Io, int DP, bool BIAS>
constexpr int kDkvWaves = (sizeof(typename Io::T) == 4 && DP > 32) || DP > 64 ? 1 : 2;

// What the two kernels hand on, and the sums of split work (splits > 1).
struct BwdParts {
  float* delta;   // [batch, heads, queries]
  float* peak;    // [batch, heads, queries]: the largest |dout| of a query (fp16 only)
  float* dq;      // [q_splits, batch, heads, queries, d]
  float* ddelta;  // [q_splits, batch, heads, queries]: parts of delta
  float *dk, *dv; // [k_splits, batch, kv_heads, keys, d]
  float* dbias;   // [buckets, heads, batch * key tiles * k_splits], or NULL
  int q_splits, k_splits;
};

// fp16: ds is formed times a power of two that brings the largest |dout| near 1, so that small gradients keep their
// bits and large ones do not overflow; 2^-floor(log2 peak), 1 for a row of zeros.
__device__ __forceinline__ float inverse_power(float peak) {
  const uint32_t e = __builtin_bit_cast(uint32_t, peak) >> 23 & 255;
  return e == 0 || e > 250 ? 1.0f : __builtin_bit_cast(float, (254 - e) << 23);
}

template <class Io, int DP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads, (kDqWaves<Io, DP, BIAS>)) void attention_dq_kernel(
    Problem a, View q, View k, View v, View o, View dout, const float* lse, View dq, BwdParts parts,
    Buckets buckets) {
  using T = typename Io::T;
  using M = Mma<Io>;
  using L = Tile<Io, DP>;
  constexpr bool kSplit = sizeof(T) == 2;
  constexpr bool kScaled = std::is_same_v<Io, F16>;
  constexpr int DC = DP / 16, DB = DP / 32, KB = kAttnKeys / 32;
  FINETUNE_DYNAMIC_LDS(attention_lds);
  T* sk = reinterpret_cast<T*>(attention_lds);
  T* sv = sk + L::bytes(kAttnKeys) / sizeof(T);
  float* line = reinterpret_cast<float*>(sv + L::bytes(kAttnKeys) / sizeof(T));

  const int tiles = (a.tq + kAttnRows - 1) / kAttnRows;
  uint32_t unit, item;
  locate(blockIdx.x, a.batch * a.kv_heads, a.group * tiles * parts.q_splits, unit, item);
  const int b = static_cast<int>(unit / a.kv_heads), kvh = static_cast<int>(unit % a.kv_heads);
  const int split = static_cast<int>(item % parts.q_splits);
  item /= parts.q_splits;
  const int tile = tiles - 1 - static_cast<int>(item % tiles);
  const int h = kvh * a.group + static_cast<int>(item / tiles);

  const int l = threadIdx.x % kWave, wave = threadIdx.x / kWave, g = l / 32;
  const int w0 = tile * kAttnRows + wave * 32, i = w0 + l % 32;
  const int off = a.tk - a.tq;
  const int64_t row0 = (int64_t(b) * a.heads + h) * a.tq;
  const float own_lse = i < a.tq ? lse[row0 + i] : -INFINITY;
  const bool live = own_lse != -INFINITY;  // a query that saw no key has no gradient

  int lo, hi;
  span_of(a, b, lo, hi);
  const auto end_of = [&](int query) { return a.causal && query + off + 1 < hi ? query + off + 1 : hi; };
  const int hi_row = end_of(i), wave_hi = end_of(w0), wave_end = end_of(w0 + 31);
  const int last = tile * kAttnRows + kAttnRows < a.tq ? tile * kAttnRows + kAttnRows : a.tq;
  const int tile_hi = end_of(last - 1);
  int k0 = lo / kAttnKeys, k1 = tile_hi > lo ? (tile_hi + kAttnKeys - 1) / kAttnKeys : k0;
  if (parts.q_splits > 1) {
    const int per = (k1 - k0 + parts.q_splits - 1) / parts.q_splits;
    k0 += split * per;
    k1 = k0 + per < k1 ? k0 + per : k1;
  }

  typename M::Frag qf[DC], df[DC];
  const int64_t ii = i < a.tq ? i : 0;
  const T *qrow = q.at<const T>(b, ii, h), *orow = o.at<const T>(b, ii, h), *drow = dout.at<const T>(b, ii, h);
  float delta = 0.0f, peak = 0.0f;
#pragma unroll
  for (int c = 0; c < DC; ++c) {
    qf[c] = row_frag<Io>(qrow, live, c, a.d);
    df[c] = row_frag<Io>(drow, live, c, a.d);
    const typename M::Frag of = row_frag<Io>(orow, live, c, a.d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      delta = fmaf(static_cast<float>(df[c][j]), static_cast<float>(of[j]), delta);
      if constexpr (kScaled) peak = fmaxf(peak, fabsf(static_cast<float>(df[c][j])));
    }
  }
  delta = halves_sum(delta);
  if constexpr (kScaled) peak = halves_max(peak);
  const float power = kScaled ? inverse_power(peak) : 1.0f;
  const float unlift = kScaled ? 0.00390625f : 1.0f;  // 2^-kLift
  const float fs = power * unlift, delta_fs = delta * fs;
  const float base = live ? kLift<Io> - own_lse * kLog2e : -INFINITY;  // p = 0

  if constexpr (BIAS) load_bias<kAttnThreads>(line, a.table, a.heads, h, buckets);

  Acc acc[DB];
#pragma unroll
  for (int n = 0; n < DB; ++n) acc[n] = zero_acc();
  float along = 0.0f;  // sum of p dp

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
#pragma unroll BIAS ? 1 : KB
    for (int n = 0; n < KB; ++n) {
      const int j0 = t * kAttnKeys + 32 * n;
      if (j0 >= wave_end) continue;
      Acc x = zero_acc(), dp = zero_acc();
      fetched_ahead<Io, 2 * DC, (kDqGroup<Io, DP, 2 * DC>)>(
          [&](int m) { return L::rows(m % 2 ? sv : sk, 32 * n, m / 2, l); },
          [&](int m, auto f) {
            if (m % 2)
              dp = M::mul(f, df[m / 2], dp);
            else
              x = M::mul(f, qf[m / 2], x);
          });
      const float* bias = line;
      float one = 0.0f;
      bool near = false;
      if constexpr (BIAS) {
        const int rel_lo = j0 - (w0 + 31) - off, rel_hi = j0 + 31 - w0 - off;
        near = rel_hi > -buckets.reach && rel_lo < buckets.reach;
        if (near) bias = line + (j0 + 4 * g - i - off + buckets.reach + kEdge);
        if (!near) one = line[rel_lo >= buckets.reach ? 2 * (buckets.reach + kEdge) : 0];
      }
      if (j0 < lo || j0 + 32 > wave_hi) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = j0 + 8 * (r / 4) + r % 4 + 4 * g;
          if (j < lo || j >= hi_row) x[r] = -INFINITY;
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int up = 8 * (r / 4) + r % 4;
        float e = fmaf(x[r], a.scale2, base);
        if constexpr (BIAS) e += near ? bias[up] : one;
        const float p = exp2_of(e);
        along = fmaf(p, dp[r], along);
        x[r] = p * fmaf(dp[r], fs, -delta_fs);
      }
      // ds as the sum of two numbers of the storage type: its rounding would add to dq's own as much again, beside
      // what o's rounding leaves in delta (error of dq 1.5 times its own rounding; so 1.2, for 15% of this kernel's time)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const typename M::Frag s = frag_of<Io>(x, 8 * c);
        typename M::Frag rest = {};
        if constexpr (kSplit) {
#pragma unroll
          for (int r = 0; r < 8; ++r) rest[r] = M::narrow(x[8 * c + r] - static_cast<float>(s[r]));
        }
        fetched_ahead<Io, DB, (kDqGroup<Io, DP, DB>)>(
            [&](int e) { return L::cols(sk, 32 * n + 16 * c, 32 * e, l); },
            [&](int e, auto f) {
              acc[e] = M::mul(f, s, acc[e]);
              if constexpr (kSplit) acc[e] = M::mul(f, rest, acc[e]);
            });
      }
    }
  }
  along = halves_sum(along);
  if (i >= a.tq) return;
  const float out_scale = a.scale / power;
  const auto value = [&](float x) { return live ? x * out_scale : 0.0f; };
  // The other kernel gets delta as the sum of p dp: o is rounded, and its error would stand in every sum over queries.
  delta = live ? along * unlift : 0.0f;
  const int64_t all = int64_t(a.batch) * a.heads * a.tq, at = row0 + i;
  if (g == 0) {
    if (parts.q_splits > 1)
      parts.ddelta[split * all + at] = delta;
    else
      parts.delta[at] = delta;
    if (kScaled && split == 0) parts.peak[at] = peak;
  }
  if (parts.q_splits > 1) {
    float* out = parts.dq + (split * all + at) * a.d;
#pragma unroll
    for (int n = 0; n < DB; ++n)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        store_four<F32>(out, 32 * n + 2 * r + 4 * g, a.d, value(acc[n][r]), value(acc[n][r + 1]),
                        value(acc[n][r + 2]), value(acc[n][r + 3]));
    return;
  }
  T* out = dq.at<T>(b, i, h);
#pragma unroll
  for (int n = 0; n < DB; ++n)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      store_four<Io>(out, 32 * n + 2 * r + 4 * g, a.d, value(acc[n][r]), value(acc[n][r + 1]),
                     value(acc[n][r + 2]), value(acc[n][r + 3]));
}

// Scores are computed queries x keys here, so that a lane has all its scores of
// one key and the probabilities are the operand of the products with dout and q.
template <class Io, int DP, bool BIAS>
__global__ __launch_bounds__(kAttnThreads, (kDkvWaves<Io, DP, BIAS>)) void attention_dkv_kernel(
    Problem a, View q, View k, View v, View dout, const float* lse, View dk, View dv, BwdParts parts,
    Buckets buckets) {
  using T = typename Io::T;
  using M = Mma<Io>;
  using L = Tile<Io, DP>;
  constexpr bool kScaled = std::is_same_v<Io, F16>, kNarrow = sizeof(T) == 4;
  constexpr int DC = DP / 16, DB = DP / 32, QN = kBwdQueries<Io, DP>, QB = QN / 32;
  FINETUNE_DYNAMIC_LDS(attention_lds);
  // two sets of tiles and of their queries' numbers in turn, so that one is written while slower waves read the other:
  // one barrier a tile (at one wave a SIMD 1010 -> 950 us on the long case; the forward, at two, 420 -> 435)
  constexpr int kTile = L::bytes(QN) / sizeof(T), kSet = kTileSet<Io, DP>;
  float* line = attention_lds + 2 * kSet;
  const Slots slots(BIAS ? buckets.reach + kEdge : 0);
  float* sums = line + (BIAS ? bias_line(buckets) : 0);  // of ds by relative position, a wave's after another's
  float* mine = sums + threadIdx.x / kWave * slots.size();
  float* block = sums + 4 * slots.size() + threadIdx.x / kWave * kBlockFloats + 32;  // the wave's

  const int tiles = (a.tk + kAttnRows - 1) / kAttnRows;
  uint32_t unit, item;
  locate(blockIdx.x, a.batch * a.kv_heads, tiles * parts.k_splits, unit, item);
  const int b = static_cast<int>(unit / a.kv_heads), kvh = static_cast<int>(unit % a.kv_heads);
  const int split = static_cast<int>(item % parts.k_splits), step = static_cast<int>(item / parts.k_splits);
  // A causal mask leaves the first tiles the most queries.  Where two workgroups share a compute unit, every other
  // round of units goes the other way, so that a long and a short one meet.
  const int tile = kDkvWaves<Io, DP, BIAS> == 2 && (unit >> 3) & 1 ? tiles - 1 - step : step;

  const int l = threadIdx.x % kWave, wave = threadIdx.x / kWave, g = l / 32;
  const int w0 = tile * kAttnRows + wave * 32, j = w0 + l % 32;
  const int off = a.tk - a.tq;
  int lo, hi;
  span_of(a, b, lo, hi);
  const bool valid = j >= lo && j < hi;
  const bool some_invalid = w0 < lo || w0 + 32 > hi;

  typename M::Frag kf[DC], vf[DC];
  const T *krow = k.at<const T>(b, valid ? j : 0, kvh), *vrow = v.at<const T>(b, valid ? j : 0, kvh);
#pragma unroll
  for (int c = 0; c < DC; ++c) {
    kf[c] = row_frag<Io>(krow, valid, c, a.d);
    vf[c] = row_frag<Io>(vrow, valid, c, a.d);
  }

  // the tiles of queries [q0, q1) see keys of this tile; (head, tile) pairs are split over workgroups
  const int t0 = tile * kAttnRows, t1 = t0 + kAttnRows;
  const int nq = (a.tq + QN - 1) / QN;
  int q0 = a.causal && t0 - off > 0 ? (t0 - off) / QN : 0;
  if (q0 > nq || t1 <= lo || t0 >= hi) q0 = nq;
  const int each = nq - q0;
  int64_t s0 = 0, s1 = int64_t(each) * a.group;
  if (parts.k_splits > 1) {
    const int64_t per = (s1 + parts.k_splits - 1) / parts.k_splits;
    s0 = split * per;
    s1 = s0 + per < s1 ? s0 + per : s1;
  }

  Acc ak[DB], av[DB];
#pragma unroll
  for (int n = 0; n < DB; ++n) ak[n] = zero_acc(), av[n] = zero_acc();
  float power = 1.0f;  // fp16: what ds is formed times
  bool first = true;
  int turn = 0;

  using Rows = Stage<Io, DP, QN, kAttnThreads>;
  Rows nx, nd;
  const bool holes = a.begin || a.end || (a.causal && off < 0);  // there may be queries that see no key
  for (int hh = 0; hh < a.group; ++hh) {
    const int64_t m0 = s0 - int64_t(hh) * each, m1 = s1 - int64_t(hh) * each;
    const int qa = q0 + static_cast<int>(m0 > 0 ? m0 : 0), qb = q0 + static_cast<int>(m1 < each ? m1 : each);
    if (!BIAS && qa >= qb) continue;
    const int h = kvh * a.group + hh;
    const int64_t at = (int64_t(b) * a.heads + h) * a.tq;
    const T *qbase = q.at<const T>(b, 0, h), *dbase = dout.at<const T>(b, 0, h);
    if constexpr (BIAS) {
      __syncthreads();
      load_bias<kAttnThreads>(line, a.table, a.heads, h, buckets);
      for (int t = threadIdx.x; t < 4 * slots.size(); t += kAttnThreads) sums[t] = 0.0f;
      __syncthreads();
    }
    float nlse = -INFINITY, ndelta = 0.0f, npeak = 0.0f, row_lse[Rows::N];
    const auto fetch_dout = [&](int t) { nd.load(dbase, dout.st, int64_t(t) * QN, 0, a.tq, a.d); };
    const auto fetch = [&](int t) {
      const int64_t i0 = int64_t(t) * QN;
      nx.load(qbase, q.st, i0, 0, a.tq, a.d);
#pragma unroll
      for (int n = 0; n < Rows::N; ++n) {
        const int64_t i = i0 + Rows::row(threadIdx.x, n);
        row_lse[n] = holes && i < a.tq ? lse[at + i] : 0.0f;
      }
      if (threadIdx.x < QN) {
        const int64_t i = i0 + threadIdx.x;
        nlse = i < a.tq ? lse[at + i] : -INFINITY;
        ndelta = i < a.tq ? parts.delta[at + i] : 0.0f;
        if constexpr (kScaled) npeak = i < a.tq ? parts.peak[at + i] : 0.0f;
      }
    };
    constexpr bool kAhead = !kBwdTight<Io, DP>;
    if (kAhead && qa < qb) fetch(qa), fetch_dout(qa);
    for (int t = qa; t < qb; ++t) {
      float* set = attention_lds + turn * kSet;
      T *sq = reinterpret_cast<T*>(set), *sd = sq + kTile;
      float *sbase = reinterpret_cast<float*>(sd + kTile), *sdelta = sbase + QN, *speak = sdelta + QN;
      turn = 1 - turn;
      if (!kAhead) fetch(t);
      const auto mend = [&](Rows& x) {  // rows of queries without a key may hold anything
        if (!holes) return;
#pragma unroll
        for (int n = 0; n < Rows::N; ++n)
          if (row_lse[n] == -INFINITY) x.zeros |= 1u << n;
      };
      mend(nx);
      nx.store(sq);
      if (!kAhead) fetch_dout(t);
      mend(nd);
      nd.store(sd);
      if (threadIdx.x < QN) {
        sbase[threadIdx.x] = nlse == -INFINITY ? -INFINITY : kLift<Io> - nlse * kLog2e;  // without a key p = 0
        sdelta[threadIdx.x] = -ndelta;
        if constexpr (kScaled) speak[threadIdx.x] = npeak;
      }
      __syncthreads();
      if (kAhead && t + 1 < qb) fetch(t + 1), fetch_dout(t + 1);
      const int i0 = t * QN;
      if constexpr (kScaled) {
        // one power of two for all of dk's sums: when a tile asks for a smaller one, the sums follow
        const float most = lanes_reduce<kWave>(speak[l % QN], [](float x, float y) { return fmaxf(x, y); });
        const float want = inverse_power(most);
        if (most > 0.0f && (first || want < power)) {
          const float ratio = want / power;
          if (!first)
#pragma unroll
            for (int n = 0; n < DB; ++n)
#pragma unroll
              for (int r = 0; r < 16; ++r) ak[n][r] *= ratio;
          power = want;
          first = false;
        }
      }
      const float unlift = kScaled ? 0.00390625f : 1.0f;
      const float fs = power * unlift;
#pragma unroll DP > 64 ? QB : 1
      for (int n = 0; n < QB; ++n) {
        const int r0 = i0 + 32 * n;
        if (a.causal && r0 + 31 + off < w0) continue;  // no query of the block sees a key of the wave
        const int lane = kNarrow ? opaque(l) : l;  // (registers)
        Acc x = zero_acc(), dp;  // dp - delta
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = 32 * n + 8 * (r / 4) + 4 * g + r % 4;
          dp[r] = sdelta[row];
        }
        if constexpr (kNarrow) {
#pragma unroll
          for (int c = 0; c < DC; ++c) {
            x = M::mul(L::rows(sq, 32 * n, c, lane), kf[c], x);
            dp = M::mul(L::rows(sd, 32 * n, c, lane), vf[c], dp);
            __builtin_amdgcn_sched_barrier(0);  // no operands loaded further ahead
          }
        } else {
          fetched_ahead<Io, 2 * DC, kAheadOf<Io, 2 * DC>>(
              [&](int m) { return L::rows(m % 2 ? sd : sq, 32 * n, m / 2, lane); },
              [&](int m, auto f) {
                if (m % 2)
                  dp = M::mul(f, vf[m / 2], dp);
                else
                  x = M::mul(f, kf[m / 2], x);
              });
        }
        const float* bias = line;
        float one = 0.0f;
        bool near = false, right = false;
        const int rel_lo = w0 - (r0 + 31) - off, rel_hi = w0 + 31 - r0 - off;
        const int place = w0 - r0 - off + buckets.reach + kEdge + static_cast<int>(threadIdx.x % 32) -
                          4 * static_cast<int>(threadIdx.x % kWave / 32);  // of the lane's first query
        if constexpr (BIAS) {
          near = rel_hi > -buckets.reach && rel_lo < buckets.reach;
          right = rel_lo >= buckets.reach;
          if (near) bias = line + place;
          if (!near) one = line[right ? 2 * (buckets.reach + kEdge) : 0];
        }
        if (some_invalid || (a.causal && r0 + off < w0 + 31)) {
          const int last = valid ? a.causal ? j - off : INT_MIN : INT_MAX;  // queries before it do not see the key
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (r0 + 8 * (r / 4) + r % 4 + 4 * g < last) x[r] = -INFINITY;
        }
        Acc ds;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int up = 8 * (r / 4) + r % 4;
          float e = fmaf(x[r], a.scale2, sbase[32 * n + up + 4 * g]);
          if constexpr (BIAS) e += near ? bias[-up] : one;
          const float p = exp2_of(e);
          x[r] = p;
          ds[r] = p * (kScaled ? dp[r] * fs : dp[r]);
        }
        if constexpr (kBwdTight<Io, DP>) __builtin_amdgcn_sched_barrier(0);
        if constexpr (BIAS) {
          const float undo = 1.0f / power;
          if (near) {
            // ds through the wave's scratch: lane t sums the diagonal key - query = t - 31 of the block
            FINETUNE_WAVE_FENCE();
#pragma unroll
            for (int r = 0; r < 16; ++r) block[(8 * (r / 4) + 4 * g + r % 4) * kBlockLine + l % 32] = ds[r];
            FINETUNE_WAVE_FENCE();
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < 32; ++r) {
              const float v = block[r * (kBlockLine + 1) + l - 31];
              s += static_cast<unsigned>(r + l - 31) < 32u ? v : 0.0f;
            }
            if (l < 63) mine[slots.at(w0 - r0 - off + l - 31)] += s * undo;
          } else {  // one bucket
            float s = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) s += ds[r];
            s = lanes_sum<kWave>(s * undo);
            FINETUNE_WAVE_FENCE();
            if (l == 0) mine[slots.at(right ? slots.most : -slots.most)] += s;
          }
        }
        if constexpr (kNarrow) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const typename M::Frag p = frag_of<Io>(x, 8 * c), s = frag_of<Io>(ds, 8 * c);
#pragma unroll
            for (int e = 0; e < DB; ++e) {
              av[e] = M::mul(L::cols(sd, 32 * n + 16 * c, 32 * e, lane), p, av[e]);
              ak[e] = M::mul(L::cols(sq, 32 * n + 16 * c, 32 * e, lane), s, ak[e]);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        } else {
          const typename M::Frag p[2] = {frag_of<Io>(x, 0), frag_of<Io>(x, 8)},
                                 s[2] = {frag_of<Io>(ds, 0), frag_of<Io>(ds, 8)};
          fetched_ahead<Io, 4 * DB, kAheadOf<Io, 4 * DB>>(
              [&](int m) { return L::cols(m % 2 ? sq : sd, 32 * n + 16 * (m / 2 / DB), 32 * (m / 2 % DB), lane); },
              [&](int m, auto f) {
                const int c = m / 2 / DB, e = m / 2 % DB;
                if (m % 2)
                  ak[e] = M::mul(f, s[c], ak[e]);
                else
                  av[e] = M::mul(f, p[c], av[e]);
              });
        }
      }
    }
    if constexpr (BIAS) {
      __syncthreads();
      if (parts.dbias) {
        const int64_t n = int64_t(a.batch) * tiles * parts.k_splits;
        const int64_t mine_at = (int64_t(b) * tiles + tile) * parts.k_splits + split;
        bucket_sums(sums, slots, kAttnThreads / kWave, buckets,
                    [&](int c, float s) { parts.dbias[(int64_t(c) * a.heads + h) * n + mine_at] = s; });
      }
    }
  }
  if (j >= a.tk) return;
  const float mk = a.scale / power, mv = kScaled ? 0.00390625f : 1.0f;
  const auto value = [&](float x, float s) { return valid ? x * s : 0.0f; };
  if (parts.k_splits > 1) {
    const int64_t place =
        (((int64_t(split) * a.batch + b) * a.kv_heads + kvh) * a.tk + j) * a.d;
#pragma unroll
    for (int n = 0; n < DB; ++n)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int x0 = 32 * n + 2 * r + 4 * g;
        store_four<F32>(parts.dk + place, x0, a.d, value(ak[n][r], mk), value(ak[n][r + 1], mk),
                        value(ak[n][r + 2], mk), value(ak[n][r + 3], mk));
        store_four<F32>(parts.dv + place, x0, a.d, value(av[n][r], mv), value(av[n][r + 1], mv),
                        value(av[n][r + 2], mv), value(av[n][r + 3], mv));
      }
    return;
  }
  T *ok = dk.at<T>(b, j, kvh), *ov = dv.at<T>(b, j, kvh);
#pragma unroll
  for (int n = 0; n < DB; ++n)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int x0 = 32 * n + 2 * r + 4 * g;
      store_four<Io>(ok, x0, a.d, value(ak[n][r], mk), value(ak[n][r + 1], mk), value(ak[n][r + 2], mk),
                     value(ak[n][r + 3], mk));
      store_four<Io>(ov, x0, a.d, value(av[n][r], mv), value(av[n][r + 1], mv), value(av[n][r + 2], mv),
                     value(av[n][r + 3], mv));
    }
}

// out[b, t, h, :] = the sum of its splits in order, for [splits, batch, heads, tokens, d]; one wave a row, two a lane.
// `first` and `second` (dk and dv) in one launch, the second's rows after the first's; with `dparts` also delta, from
// its parts.
struct SumJob {
  const float* part;
  View out;
};
template <class Io>
__global__ __launch_bounds__(kWave) void attention_sum_kernel(SumJob first, SumJob second, int splits, int64_t rows,
                                                              int heads, int tokens, int d, const float* dparts,
                                                              float* delta) {
  using T = typename Io::T;
  const bool other = blockIdx.x >= rows;
  const int64_t row = other ? blockIdx.x - rows : blockIdx.x, t = row % tokens, bh = row / tokens;
  T* to = other ? second.out.at<T>(bh / heads, t, bh % heads) : first.out.at<T>(bh / heads, t, bh % heads);
  const float* part = (other ? second.part : first.part) + row * d;
  const int l = threadIdx.x;
  float x = 0.0f, y = 0.0f;
#pragma unroll 8
  for (int n = 0; n < splits; ++n) {
    const float* from = part + n * rows * d;
    if (l < d) x += from[l];
    if (l + kWave < d) y += from[l + kWave];
  }
  if (l < d) to[l] = Io::narrow(x);
  if (l + kWave < d) to[l + kWave] = Io::narrow(y);
  if (dparts && l == 0) {
    float s = 0.0f;
    for (int n = 0; n < splits; ++n) s += dparts[n * rows + row];
    delta[row] = s;
  }
}

}  // namespace finetune
