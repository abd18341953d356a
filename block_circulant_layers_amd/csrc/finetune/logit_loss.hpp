// logit_loss.hpp -- token log-probabilities, the preference loss and the
// clipped policy loss on vocabulary logits, with the logits' gradient.
//
// Per position: lse = log sum_j exp x_j, logp = x[label] - lse.  Every loss
// here is a function of the positions' logp, so its logits' gradient is
//   dx_j = g (1[j = label] - exp(x_j - lse)),  g = d loss / d logp.
#pragma once

#include "device.hpp"

namespace finetune {

constexpr int kLogitThreads = 256;
constexpr int64_t kIgnore = -100;

// Logits as the kernels see them: row r = (sequence r / positions, position
// r % positions), both below 2^31.
template <class Io>
struct Rows {
  typename Io::T* data;
  int64_t seq_stride, pos_stride;
  __device__ __forceinline__ typename Io::T* row(int64_t r, int64_t positions) const {
    const uint32_t n = static_cast<uint32_t>(positions), q = static_cast<uint32_t>(r) / n;
    return data + q * seq_stride + (static_cast<uint32_t>(r) - q * n) * static_cast<int64_t>(pos_stride);
  }
};

constexpr float kLog2eHi = 1.44269502162933349609375f;
constexpr float kLog2eLo = 1.925963033500011e-8f;  // log2(e) - kLog2eHi

// exp(d) for d <= 0 through the hardware's exp2.  log2(e) is taken as a sum of
// two floats: its rounding alone (1.3e-8) would shift every exponential, and
// with it every log-probability, the same way, which a sum over a sequence's
// positions does not average out.
__device__ __forceinline__ float exp_of(float d) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(d, kLog2eHi, d * kLog2eLo));
}

__device__ __forceinline__ float max_of(float a, float b) { return a > b ? a : b; }

// the largest of n values and `top`, n even
template <int N>
__device__ __forceinline__ float max_over(const float (&x)[N], float top) {
  static_assert(N % 2 == 0);
  float a[2] = {top, top};
#pragma unroll
  for (int i = 0; i < N; i += 2) FINETUNE_MAX3(a[i / 2 % 2], x[i], x[i + 1], a[i / 2 % 2]);
  return max_of(a[0], a[1]);
}

// A running maximum m of values seen and s = the sum of exp(x - m); NaN values
// make s NaN, values of -inf alone leave m = -inf and s = 0.
struct MaxSum {
  float m = -INFINITY, s = 0.0f;
  static __device__ __forceinline__ float base(float top) { return top == -INFINITY ? 0.0f : top; }
  // n values at once: one rescaling for all of them
  template <int N>
  __device__ __forceinline__ void add(const float (&x)[N]) {
    const float top = max_over(x, m);
    const float b = base(top);
    s *= exp_of(m - b);
    m = top;
    float a[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) a[i % 2] += exp_of(x[i] - b);
    s += a[0] + a[1];
  }
  __device__ __forceinline__ void join(float om, float os) {
    const float top = max_of(om, m), b = base(top);
    s = s * exp_of(m - b) + os * exp_of(om - b);
    m = top;
  }
  // over the NT threads of a workgroup, the result in every thread; `sm` holds
  // 2 NT / 64 slots and may be reused after the next barrier
  template <int NT>
  __device__ __forceinline__ void join_group(float* sm) {
    const float top = lanes_reduce<kWave>(m, [](float a, float b) { return max_of(a, b); });
    s = lanes_sum<kWave>(s * exp_of(m - base(top)));
    m = top;
    if constexpr (NT > kWave) {
      constexpr int W = NT / kWave;
      if (threadIdx.x % kWave == 0) {
        sm[threadIdx.x / kWave] = m;
        sm[W + threadIdx.x / kWave] = s;
      }
      __syncthreads();
      float all = sm[0];
#pragma unroll
      for (int i = 1; i < W; ++i) all = max_of(all, sm[i]);
      const float b = base(all);
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) t += sm[W + i] * exp_of(sm[i] - b);
      m = all;
      s = t;
    }
  }
  // log sum exp; NaN for a row whose maximum is infinite (its softmax has no value)
  __device__ __forceinline__ double lse() const { return m + log(static_cast<double>(s)) + (m - m); }
};

// Maximum and sum of the columns [begin, end) of a row by NT threads, four
// 16-byte pieces of a thread in flight.
template <class Io, int NT, bool STREAM>
__device__ __forceinline__ MaxSum row_max_sum(const typename Io::T* x, int begin, int end) {
  constexpr int V = Io::kVec, U = 4;
  const Pieces<Io> p(x, begin, end);
  MaxSum a;
  int j = p.first + static_cast<int>(threadIdx.x) * V;
  const auto batch = [&](auto n) {
    constexpr int B = decltype(n)::value;
    typename Io::Vec raw[B];
#pragma unroll
    for (int u = 0; u < B; ++u) raw[u] = load_vec<Io, STREAM>(x + j + u * NT * V);
    float f[B * V];
#pragma unroll
    for (int k = 0; k < B * V; ++k) f[k] = Io::widen(raw[k / V][k % V]);
    a.add(f);
    j += B * NT * V;
  };
  while (j + (U - 1) * NT * V < p.last) batch(std::integral_constant<int, U>{});
  if (j + NT * V < p.last) batch(std::integral_constant<int, 2>{});  // up to three are left
  if (j < p.last) batch(std::integral_constant<int, 1>{});
  p.template rest<NT>([&](int c) {
    const float f[2] = {Io::widen(x[c]), -INFINITY};
    a.add(f);
  });
  return a;
}

// lse and logp of every position.  One workgroup per row (parts = 1), or, where
// there are fewer rows than the chip has room for, `parts` workgroups of `per`
// columns each, whose maxima and sums go to `partial` for the next kernel to
// join, and the label's logit to `picked`: the next kernel may replace it.
// STREAM: rows below `keep` are read past the caches, the others through
// them.
template <class Io, int NT, bool STREAM>
__global__ void __launch_bounds__(NT)
    token_logprob_kernel(Rows<Io> in, const int64_t* labels, float* logp, float* lse, float2* partial,
                         float* picked, int64_t rows, int64_t positions, int v, int parts, int per, int64_t keep) {
  __shared__ float sm[2 * NT / kWave + 1];
  for (int64_t i = blockIdx.x; i < rows * parts; i += gridDim.x) {
    const int64_t r = parts == 1 ? i : static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(parts));
    const int64_t label = labels[r];
    if (label < 0 || label >= v) {
      if (parts == 1 && threadIdx.x == 0) logp[r] = lse[r] = label == kIgnore ? 0.0f : NAN;
      continue;
    }
    const typename Io::T* x = in.row(r, positions);
    const int begin = static_cast<int>(i - r * parts) * per, end = begin + per < v ? begin + per : v;
    MaxSum a = STREAM && r < keep ? row_max_sum<Io, NT, STREAM>(x, begin, end)
                                  : row_max_sum<Io, NT, false>(x, begin, end);
    a.template join_group<NT>(sm);
    if (threadIdx.x == 0) {
      if (parts > 1) {
        partial[i] = make_float2(a.m, a.s);
        if (label >= begin && label < end) picked[r] = Io::widen(x[label]);
      } else {
        const double l = a.lse();
        lse[r] = static_cast<float>(l);
        logp[r] = static_cast<float>(Io::widen(x[label]) - l);
      }
    }
    if (NT > kWave) __syncthreads();
  }
}

// The positions' lse and logp from their parts.
template <class Io>
struct JoinParts {
  Rows<Io> in;
  const float2* partial;  // null: logp and lse are there already
  const float* picked;
  float* lse;
  int parts, lanes, v;  // lanes: of one row, a power of two up to 64

  // logp of row r by `lanes` threads in a row, each calling this with its index
  // `lane` among them (r the same; label kIgnore where there is no row); lane 0
  // has the result, and stores it and lse if `write`.  (One thread a row took
  // 8.6 us for the 64 parts of a single row.)
  __device__ __forceinline__ float row(int64_t r, int lane, int64_t label, float* logp, bool write,
                                       float* lse_out = nullptr) const {
    if (!partial) {
      if (lse_out) *lse_out = label == kIgnore ? 0.0f : lse[r];
      return label == kIgnore ? 0.0f : logp[r];
    }
    const bool known = label >= 0 && label < v;
    MaxSum a;
    if (known)
      for (int k = lane; k < parts; k += lanes) {
        const float2 q = partial[r * parts + k];
        a.join(q.x, q.y);
      }
    for (int o = lanes / 2; o > 0; o /= 2) a.join(__shfl_xor(a.m, o, kWave), __shfl_xor(a.s, o, kWave));
    if (lane != 0) return 0.0f;
    const double l = known ? a.lse() : label == kIgnore ? 0.0 : NAN;
    const float p = static_cast<float>(known ? picked[r] - l : l);
    if (lse_out) *lse_out = static_cast<float>(l);
    if (write) {
      lse[r] = static_cast<float>(l);
      logp[r] = p;
    }
    return p;
  }

  // f(row, label, logp) for rows [first, first + count), by lane 0 of each row's
  // threads among the NT of a workgroup
  template <int NT, class F>
  __device__ __forceinline__ void rows(int64_t first, int64_t count, const int64_t* labels, float* logp, bool write,
                                       F f) const {
    const int lane = static_cast<int>(threadIdx.x) & (lanes - 1), at_once = NT / lanes;
    for (int64_t base = 0; base < count; base += at_once) {
      const int64_t i = base + static_cast<int>(threadIdx.x) / lanes, r = first + i;
      const int64_t label = i < count ? labels[r] : kIgnore;
      const float p = row(r, lane, label, logp, write && i < count);
      if (lane == 0 && i < count) f(r, label, p);
    }
  }
};

// ... for a caller that wants nothing but the log-probabilities
constexpr int kJoinRows = 64;  // of a workgroup
template <class Io>
__global__ void __launch_bounds__(kLogitThreads)
    join_kernel(JoinParts<Io> join, const int64_t* labels, float* logp, int64_t rows) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kJoinRows;
  join.template rows<kLogitThreads>(first, rows - first < kJoinRows ? rows - first : kJoinRows, labels, logp, true,
                                    [](int64_t, int64_t, float) {});
}

// One row's gradient g (1[j = label] - exp(x_j - lse)).  x - lse is taken first:
// it is small wherever the softmax is not, so its rounding and the rounding of
// log2(e) cost 2.5 |x - lse| units of 2^-24 whatever offset the row has, and a
// row of any finite values has a finite gradient.  (One multiply-add instead, x
// log2(e) against a rounded lse log2(e) with the rest in g's factor, saves an
// instruction an element, which shows where a row's exponentials are not hidden
// behind its bytes: a policy step of 16384 rows of 8000 fp16 118 us, 122 us so,
// of 8192 rows of 131072 bf16 658 us both.  But it takes its error from x: 1.3e-4
// of every softmax value at logits near 1e4, NaN past 1e10.)
struct RowGrad {
  float g, lse;
  int label;
  __device__ __forceinline__ RowGrad(float g_, float lse_, int label_) : g(g_), lse(lse_), label(label_) {}
  __device__ __forceinline__ float at(float x) const {
    return -g * __builtin_amdgcn_exp2f((x - lse) * kLog2eHi);
  }
  template <class Io>
  __device__ __forceinline__ typename Io::Vec piece(typename Io::Vec x, int j) const {
    typename Io::Vec o;
#pragma unroll
    for (int k = 0; k < Io::kVec; ++k) o[k] = Io::narrow(at(Io::widen(x[k])));
    if (static_cast<unsigned>(label - j) < static_cast<unsigned>(Io::kVec)) {
#pragma unroll
      for (int k = 0; k < Io::kVec; ++k)
        if (label == j + k) o[k] = Io::narrow(g + at(Io::widen(x[k])));
    }
    return o;
  }
};

// The gradient's factor of every row: up[...] * slope[...].
struct RowScale {
  const float* up;     // may be null (then `scale`)
  const float* slope;  // never null
  float scale;
  int64_t up_n;        // up is indexed by sequence modulo up_n
  bool slope_by_row;   // slope by row, else by sequence
  __device__ __forceinline__ float at(int64_t r, int64_t positions) const {
    const uint32_t seq = static_cast<uint32_t>(r) / static_cast<uint32_t>(positions);
    return (up ? up[seq % static_cast<uint32_t>(up_n)] : scale) * slope[slope_by_row ? r : seq];
  }
};

// Columns [begin, end) of a row's gradient by NT threads; `x` and `o` are the
// rows of the logits and of the gradient.
template <class Io, int NT, bool STREAM>
__device__ __forceinline__ void write_zeros(typename Io::T* o, int begin, int end) {
  const Pieces<Io> p(o, begin, end);
  for (int j = p.first + static_cast<int>(threadIdx.x) * Io::kVec; j < p.last; j += NT * Io::kVec)
    store_vec<Io, STREAM>(o + j, typename Io::Vec{});
  p.template rest<NT>([&](int c) { o[c] = 0; });
}
template <class Io, int NT, bool STREAM>
__device__ __forceinline__ void write_grad(const RowGrad& grad, const typename Io::T* x, typename Io::T* o, int begin,
                                           int end) {
  constexpr int V = Io::kVec, U = 4;
  const Pieces<Io> p(o, begin, end);  // aligned stores; the loads too where both rows lie alike
  int j = p.first + static_cast<int>(threadIdx.x) * V;
  for (; j + (U - 1) * NT * V + V <= p.last; j += U * NT * V) {
    typename Io::Vec raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = load_vec<Io, STREAM>(x + j + u * NT * V);
#pragma unroll
    for (int u = 0; u < U; ++u) store_vec<Io, STREAM>(o + j + u * NT * V, grad.piece<Io>(raw[u], j + u * NT * V));
  }
  for (; j < p.last; j += NT * V) store_vec<Io, STREAM>(o + j, grad.piece<Io>(load_vec<Io, STREAM>(x + j), j));
  p.template rest<NT>([&](int c) {
    const float q = grad.at(Io::widen(x[c]));
    o[c] = Io::narrow(c == grad.label ? grad.g + q : q);
  });
}

// The gradient of every row, `parts` workgroups of `per` columns a row, the
// last row first: a step's logits were read just before, and the last of them
// are still in the 256 MB cache.
template <class Io, int NT, bool STREAM>
__global__ void __launch_bounds__(NT)
    logits_grad_kernel(Rows<Io> in, const int64_t* labels, const float* lse, RowScale scale, Rows<Io> out,
                       int64_t rows, int64_t positions, int v, int parts, int per) {
  for (int64_t n = blockIdx.x; n < rows * parts; n += gridDim.x) {
    const int64_t i = rows * parts - 1 - n;
    const int64_t r = parts == 1 ? i : static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(parts));
    const int begin = static_cast<int>(i - r * parts) * per, end = begin + per < v ? begin + per : v;
    const int64_t label = labels[r];
    typename Io::T* o = out.row(r, positions);
    if (label == kIgnore) {
      write_zeros<Io, NT, STREAM>(o, begin, end);
      continue;
    }
    const bool known = label >= 0 && label < v;
    const RowGrad grad(known ? scale.at(r, positions) : NAN, lse[r], known ? static_cast<int>(label) : -1);
    write_grad<Io, NT, STREAM>(grad, in.row(r, positions), o, begin, end);
  }
}

struct Preference {
  int kind;
  bool average;
  double beta, smoothing;
};

// A pair's loss, log-ratios and slopes, in every thread of a workgroup of NT.
// The sums run in fp64 (a few values per thread), all four of them through one
// barrier; `s` may be reused after the next one.
struct Pair {
  double loss, ratio[2], slope[2];
};
template <class Io, int NT>
__device__ __forceinline__ Pair pair_of(const JoinParts<Io>& join, const int64_t* labels, float* logp, const float* ref,
                                        const Preference& how, int64_t b, int64_t pairs, int64_t positions, bool write,
                                        double (&s)[4][NT / kWave]) {
  constexpr int W = NT / kWave;
  double sum[4] = {};  // log-ratio and count of the chosen sequence, then of the rejected one
  if (!join.partial) {
    // all loads of a round at once, masked positions' too
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < positions; i += NT) {
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int64_t r = (b + side * pairs) * positions + i, label = labels[r];
        const double p = logp[r], q = ref[r];
        sum[2 * side] += label == kIgnore ? 0.0 : p - q;
        sum[2 * side + 1] += label == kIgnore ? 0.0 : 1.0;
      }
    }
  } else {
#pragma unroll
    for (int side = 0; side < 2; ++side)
      join.template rows<NT>((b + side * pairs) * positions, positions, labels, logp, write,
                             [&](int64_t r, int64_t label, float p) {
                               if (label == kIgnore) return;
                               sum[2 * side] += static_cast<double>(p) - static_cast<double>(ref[r]);
                               sum[2 * side + 1] += 1.0;
                             });
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    sum[k] = lanes_sum<kWave>(sum[k]);
    if (threadIdx.x % kWave == 0) s[k][threadIdx.x / kWave] = sum[k];
  }
  __syncthreads();
  Pair q;
  double count[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    double a = 0.0, c = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      a += s[2 * side][w];
      c += s[2 * side + 1][w];
    }
    count[side] = how.average && c > 0.0 ? c : 1.0;
    q.ratio[side] = a / count[side];
  }
  const double h = q.ratio[0] - q.ratio[1], z = how.beta * h, e = how.smoothing;
  double dh;
  if (how.kind == 0) {
    const double t = exp(-fabs(z)), low = log1p(t);
    const double up = (z < 0.0 ? z : 0.0) - low, down = (z > 0.0 ? -z : 0.0) - low;  // log sigma(z) and log sigma(-z)
    const double big = 1.0 / (1.0 + t), small = t * big;                             // sigma(|z|) and sigma(-|z|)
    q.loss = -(1.0 - e) * up - (e > 0.0 ? e * down : 0.0);  // both may be infinite
    dh = z < 0.0 ? -how.beta * ((1.0 - e) * big - e * small) : -how.beta * ((1.0 - e) * small - e * big);
  } else if (how.kind == 1) {
    q.loss = z < 1.0 ? 1.0 - z : z >= 1.0 ? 0.0 : z;  // the last: NaN
    dh = z < 1.0 ? -how.beta : z >= 1.0 ? 0.0 : z;
  } else {
    const double gap = h - 0.5 / how.beta;
    q.loss = gap * gap;
    dh = 2.0 * gap;
  }
  q.slope[0] = dh / count[0];
  q.slope[1] = -dh / count[1];
  return q;
}

struct PreferenceOut {
  float *loss, *logratio, *slope;
  __device__ __forceinline__ void store(const Pair& q, int64_t b, int64_t pairs) const {
    if (threadIdx.x != 0) return;
    loss[b] = static_cast<float>(q.loss);
    logratio[b] = static_cast<float>(q.ratio[0]);
    logratio[b + pairs] = static_cast<float>(q.ratio[1]);
    slope[b] = static_cast<float>(q.slope[0]);
    slope[b + pairs] = static_cast<float>(q.slope[1]);
  }
};

// One workgroup a pair, of 1024 threads because its loads wait for each other (4
// pairs of 2 x 1024 positions: 7.8 us, with 256 threads 10.8 us).
constexpr int kPairThreads = 1024;
template <class Io>
__global__ void __launch_bounds__(kPairThreads)
    preference_kernel(JoinParts<Io> join, const int64_t* labels, float* logp, const float* ref, Preference how,
                      PreferenceOut out, int64_t pairs, int64_t positions) {
  __shared__ double s[4][kPairThreads / kWave];
  for (int64_t b = blockIdx.x; b < pairs; b += gridDim.x) {
    out.store(pair_of<Io, kPairThreads>(join, labels, logp, ref, how, b, pairs, positions, true, s), b, pairs);
    __syncthreads();
  }
}

// The step's second and last launch where there are few rows: every workgroup
// works its pair's slope out for itself and writes its part of a row's
// gradient, and one more a pair writes the pair's results.  A launch more costs the
// host 5 us (a pair of 16 x 1009 fp32: 14.4 us with it, 10.5 us so).
template <class Io>
__global__ void __launch_bounds__(kLogitThreads)
    preference_grad_kernel(JoinParts<Io> join, const int64_t* labels, float* logp, const float* ref, Preference how,
                           float scale, PreferenceOut res, Rows<Io> out, int64_t pairs, int64_t positions, int parts,
                           int per) {
  constexpr int NT = kLogitThreads;
  __shared__ double s[4][NT / kWave];
  __shared__ float told;
  if (blockIdx.x < pairs) {
    res.store(pair_of<Io, NT>(join, labels, logp, ref, how, blockIdx.x, pairs, positions, true, s), blockIdx.x, pairs);
    return;
  }
  const uint32_t i = blockIdx.x - static_cast<uint32_t>(pairs), r = i / static_cast<uint32_t>(parts);
  const int begin = static_cast<int>(i - r * parts) * per, end = begin + per < join.v ? begin + per : join.v;
  const int64_t label = labels[r];
  typename Io::T* o = out.row(r, positions);
  if (label == kIgnore) {
    write_zeros<Io, NT, false>(o, begin, end);
    return;
  }
  const uint32_t seq = r / static_cast<uint32_t>(positions);
  const bool chosen = seq < pairs;
  const Pair q = pair_of<Io, NT>(join, labels, logp, ref, how, chosen ? seq : seq - pairs, pairs, positions, false, s);
  float lse = 0.0f;
  const int lane = static_cast<int>(threadIdx.x);
  if (lane < kWave) {  // one wave: this row's lse from its parts
    join.row(r, lane < join.lanes ? lane : join.parts, label, logp, false, &lse);
    if (lane == 0) told = lse;
  }
  __syncthreads();
  const bool known = label >= 0 && label < join.v;
  const float slope = static_cast<float>(chosen ? q.slope[0] : q.slope[1]);
  const RowGrad grad(known ? scale * slope : NAN, told, known ? static_cast<int>(label) : -1);
  write_grad<Io, NT, false>(grad, join.in.row(r, positions), o, begin, end);
}

struct Policy {
  int reduction;
  double low, high, kl;
};

struct PolicyTerm {
  double loss, kl, slope;
};

// One position's loss, KL and d loss / d logp.
__device__ __forceinline__ PolicyTerm policy_term(const Policy& how, double logp, double old, bool with_ref, double ref,
                                                  double adv) {
  PolicyTerm t{};
  const double r = exp(logp - old), lo = 1.0 - how.low, hi = 1.0 + how.high;
  const double held = (r < lo ? lo : r > hi ? hi : r) * adv, free = r * adv;
  t.loss = free > held ? -held : -free;  // a NaN ratio makes `free` NaN and stays
  t.slope = free > held ? 0.0 : -free;
  if (with_ref) {
    const double q = ref - logp, e = expm1(q);
    t.kl = e - q;
    t.loss += how.kl * t.kl;
    t.slope -= how.kl * e;
  }
  return t;
}

// What a position counts in the reduced loss.
struct PolicyWeight {
  const int* counts;  // unmasked positions of every sequence (POLICY_SEQUENCE_MEAN)
  const int* total;   // ... of all (POLICY_TOKEN_MEAN)
  int reduction;
  int64_t seqs;
  __device__ __forceinline__ int count(int64_t seq) const {
    return reduction == 0 ? total[0] : reduction == 1 ? counts[seq] : 1;
  }
  __device__ __forceinline__ double of(int count) const {
    return 1.0 / (static_cast<double>(count) * (reduction == 1 ? static_cast<double>(seqs) : 1.0));
  }
};

struct PolicyInputs {
  const float *old, *ref, *adv;  // ref may be null
  bool per_token;
};

constexpr int kPolicyThreads = 1024;

// The counts that the reduction needs, by one workgroup of NT: all positions at
// once, or a wave for a sequence at a time.
template <int NT>
__device__ __forceinline__ void policy_counts(const int64_t* labels, int* counts, int* total, int reduction,
                                              int64_t seqs, int64_t positions, int* s) {
  if (reduction == 0) {
    int c = 0;
#pragma unroll 8
    for (int64_t r = threadIdx.x; r < seqs * positions; r += NT) c += labels[r] != kIgnore;
    c = block_sum<NT>(c, s);
    if (threadIdx.x == 0) total[0] = c;
  } else if (reduction == 1) {
    const int lane = threadIdx.x % kWave;
    for (int64_t q = threadIdx.x / kWave; q < seqs; q += NT / kWave) {
      int c = 0;
#pragma unroll 8
      for (int64_t i = lane; i < positions; i += kWave) c += labels[q * positions + i] != kIgnore;
      c = lanes_sum<kWave>(c);
      if (lane == 0) counts[q] = c;
    }
  }
}

__global__ void __launch_bounds__(kPolicyThreads)
    policy_count_kernel(const int64_t* labels, int* counts, int* total, int reduction, int64_t seqs,
                        int64_t positions) {
  __shared__ int s[kPolicyThreads / kWave];
  policy_counts<kPolicyThreads>(labels, counts, total, reduction, seqs, positions, s);
}

// A position's slope and its shares of the loss and the KL.
struct PolicyShare {
  float slope = 0.0f;
  double2 share = make_double2(0.0, 0.0);
};
__device__ __forceinline__ PolicyShare policy_share(const Policy& how, const PolicyInputs& in, double weight, int64_t r,
                                                    int64_t seq, float logp) {
  const PolicyTerm e = policy_term(how, logp, in.old[r], in.ref != nullptr, in.ref ? in.ref[r] : 0.0f,
                                   in.adv[in.per_token ? r : seq]);
  return {static_cast<float>(weight * e.slope), make_double2(weight * e.loss, weight * e.kl)};
}

// Every position's logp, lse and slope, and the reduced loss and KL, by one
// workgroup of NT.
template <class Io, int NT>
__device__ __forceinline__ void policy_all(const JoinParts<Io>& join, const int64_t* labels, float* logp,
                                           const PolicyInputs& in, const PolicyWeight& weight, int* counts, int* total,
                                           const Policy& how, float* stats, float* slope, int64_t seqs,
                                           int64_t positions, int (&sc)[NT / kWave], double (&s)[2][NT / kWave]) {
  policy_counts<NT>(labels, counts, total, how.reduction, seqs, positions, sc);
  __syncthreads();
  const uint32_t n = static_cast<uint32_t>(positions);
  double a = 0.0, k = 0.0;
  join.template rows<NT>(0, seqs * positions, labels, logp, true, [&](int64_t r, int64_t label, float p) {
    PolicyShare e;
    const uint32_t seq = static_cast<uint32_t>(r) / n;
    if (label != kIgnore) e = policy_share(how, in, weight.of(weight.count(seq)), r, seq, p);
    slope[r] = e.slope;
    a += e.share.x;
    k += e.share.y;
  });
  a = block_sum<NT>(a, s[0]);
  k = block_sum<NT>(k, s[1]);
  if (threadIdx.x == 0) {
    stats[0] = static_cast<float>(a);
    stats[1] = static_cast<float>(k);
  }
}

template <class Io>
__global__ void __launch_bounds__(kPolicyThreads)
    policy_kernel(JoinParts<Io> join, const int64_t* labels, float* logp, PolicyInputs in, PolicyWeight weight,
                  int* counts, int* total, Policy how, float* stats, float* slope, int64_t seqs, int64_t positions) {
  __shared__ double s[2][kPolicyThreads / kWave];
  __shared__ int sc[kPolicyThreads / kWave];
  policy_all<Io, kPolicyThreads>(join, labels, logp, in, weight, counts, total, how, stats, slope, seqs, positions, sc,
                                 s);
}

// The same for many rows, none of them in parts: a thread a row, whose shares go
// to `terms` for policy_sum_kernel, after policy_count_kernel.
__global__ void __launch_bounds__(kLogitThreads)
    policy_rows_kernel(const int64_t* labels, const float* logp, PolicyInputs in, PolicyWeight weight, Policy how,
                       float* slope, double2* terms, int64_t rows, int64_t positions) {
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kLogitThreads + threadIdx.x; r < rows;
       r += static_cast<int64_t>(gridDim.x) * kLogitThreads) {
    PolicyShare e;
    const uint32_t seq = static_cast<uint32_t>(r) / static_cast<uint32_t>(positions);
    if (labels[r] != kIgnore) e = policy_share(how, in, weight.of(weight.count(seq)), r, seq, logp[r]);
    slope[r] = e.slope;
    terms[r] = e.share;
  }
}

// The step's second and last launch where there are few rows: every workgroup
// works its row's slope out for itself and writes its part of the gradient, the
// first one everything else (4 x 8 x 32768 half: 14.6 us with a launch between,
// 10.8 us so).
template <class Io>
__global__ void __launch_bounds__(kLogitThreads)
    policy_grad_kernel(JoinParts<Io> join, const int64_t* labels, float* logp, PolicyInputs in, PolicyWeight weight,
                       int* counts, int* total, Policy how, float scale, float* stats, float* slope, Rows<Io> out,
                       int64_t seqs, int64_t positions, int parts, int per) {
  constexpr int NT = kLogitThreads;
  __shared__ double s[2][NT / kWave];
  __shared__ int sc[NT / kWave];
  __shared__ float told[2];
  if (blockIdx.x == 0) {
    policy_all<Io, NT>(join, labels, logp, in, weight, counts, total, how, stats, slope, seqs, positions, sc, s);
    return;
  }
  const uint32_t i = blockIdx.x - 1, r = i / static_cast<uint32_t>(parts), n = static_cast<uint32_t>(positions);
  const int begin = static_cast<int>(i - r * parts) * per, end = begin + per < join.v ? begin + per : join.v;
  const int64_t label = labels[r];
  typename Io::T* o = out.row(r, positions);
  if (label == kIgnore) {
    write_zeros<Io, NT, false>(o, begin, end);
    return;
  }
  const uint32_t seq = r / n;
  int c = 0;
  if (how.reduction != 2) {
    const int64_t first = how.reduction == 0 ? 0 : static_cast<int64_t>(seq) * n, last = how.reduction == 0 ? seqs * n : first + n;
    for (int64_t k = first + threadIdx.x; k < last; k += NT) c += labels[k] != kIgnore;
    c = block_sum<NT>(c, sc);
  }
  const int lane = static_cast<int>(threadIdx.x);
  if (lane < kWave) {  // one wave: this row from its parts
    float lse = 0.0f;
    const float p = join.row(r, lane < join.lanes ? lane : join.parts, label, logp, false, &lse);
    if (lane == 0) {
      told[0] = lse;
      told[1] = scale * policy_share(how, in, weight.of(how.reduction == 2 ? 1 : c), r, seq, p).slope;
    }
  }
  __syncthreads();
  const bool known = label >= 0 && label < join.v;
  const RowGrad grad(known ? told[1] : NAN, told[0], known ? static_cast<int>(label) : -1);
  write_grad<Io, NT, false>(grad, join.in.row(r, positions), o, begin, end);
}

// The positions' shares summed in a fixed order.
__global__ void __launch_bounds__(kPolicyThreads)
    policy_sum_kernel(const double2* terms, float* stats, int64_t rows) {
  __shared__ double s[2][kPolicyThreads / kWave];
  double a = 0.0, k = 0.0;
#pragma unroll 8
  for (int64_t r = threadIdx.x; r < rows; r += kPolicyThreads) {
    const double2 t = terms[r];
    a += t.x;
    k += t.y;
  }
  a = block_sum<kPolicyThreads>(a, s[0]);
  k = block_sum<kPolicyThreads>(k, s[1]);
  if (threadIdx.x == 0) {
    stats[0] = static_cast<float>(a);
    stats[1] = static_cast<float>(k);
  }
}

// A position's log-probability, loss share, slope and gradient with its logits
// read once: one workgroup holds the row in registers, R 16-byte pieces a
// thread, and one more column a thread for what lies outside the pieces.  With
// 8192 rows of 131072 bf16, 5808 of them unmasked, it moves 3.7 GB in 660 us;
// a copy by workgroups of this shape reaches 6.1 TB/s (600 us).
template <class Io, int NT, int R, bool STREAM>
__global__ void __launch_bounds__(NT, 4)  // 128 registers: 16 waves a compute unit
    policy_step_kernel(Rows<Io> in, const int64_t* labels, PolicyInputs inputs, PolicyWeight weight, Policy how,
                       float scale, float* logp, float* lse, float* slope, double2* terms, Rows<Io> out,
                       int64_t positions, int v) {
  constexpr int V = Io::kVec;
  __shared__ float sm[2 * NT / kWave];
  __shared__ float told[2];
  const int64_t r = blockIdx.x;
  const int64_t label = labels[r];
  typename Io::T* o = out.row(r, positions);
  if (label < 0 || label >= v) {
    // masked: zeros; a label out of range: NaN
    const float fill = label == kIgnore ? 0.0f : NAN;
    typename Io::Vec f;
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = Io::narrow(fill);
    const Pieces<Io> p(o, 0, v);
    for (int j = p.first + static_cast<int>(threadIdx.x) * V; j < p.last; j += NT * V) store_vec<Io, STREAM>(o + j, f);
    p.template rest<NT>([&](int c) { o[c] = f[0]; });
    if (threadIdx.x == 0) {
      logp[r] = lse[r] = slope[r] = fill;
      terms[r] = make_double2(fill, fill);
    }
    return;
  }
  const typename Io::T* x = in.row(r, positions);
  const Pieces<Io, NT == kWave ? 16 : 128> p(o, 0, v);  // at most NT columns outside the pieces
  // the single values first, converted later: loads return in order, so a use of
  // the last one issued would wait for all
  int column = -1;
  p.template rest<NT>([&](int c) { column = c; });
  const typename Io::T extra_stored = x[column >= 0 ? column : 0], picked_stored = x[label];
  const uint32_t seq = static_cast<uint32_t>(r) / static_cast<uint32_t>(positions);
  const float old = inputs.old[r], ref = inputs.ref ? inputs.ref[r] : 0.0f,
              adv = inputs.adv[inputs.per_token ? r : seq];
  const int count = weight.count(seq);
  typename Io::Vec raw[R] = {};
  int j = p.first + static_cast<int>(threadIdx.x) * V;
  // no branch between the loads, or every use would wait for all of them: past
  // the last piece a thread loads that one again, and sets it aside below
  if (p.last > p.first) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int at = j + i * NT * V;
      raw[i] = load_vec<Io, STREAM>(x + (at < p.last ? at : p.last - V));
    }
  }

  // the exponentials of a batch of pieces while the next ones are on their way
  MaxSum a;
  constexpr int B = 4;
#pragma unroll
  for (int i = 0; i < R; i += B) {
    float f[B * V];
#pragma unroll
    for (int q = 0; q < B; ++q) {
      const bool there = j + (i + q) * NT * V < p.last;
#pragma unroll
      for (int k = 0; k < V; ++k) f[q * V + k] = there ? Io::widen(raw[i + q][k]) : -INFINITY;
    }
    a.add(f);
  }
  const float extra = column >= 0 ? Io::widen(extra_stored) : -INFINITY, picked = Io::widen(picked_stored);
  const float edge[2] = {extra, -INFINITY};
  a.add(edge);
  a.template join_group<NT>(sm);
  if (threadIdx.x == 0) {
    const double l = a.lse();
    const float lp = static_cast<float>(picked - l);
    const PolicyTerm e = policy_term(how, lp, old, inputs.ref != nullptr, ref, adv);
    const double w = weight.of(count);
    const float g = static_cast<float>(w * e.slope);
    lse[r] = told[0] = static_cast<float>(l);
    told[1] = scale * g;
    logp[r] = lp;
    slope[r] = g;
    terms[r] = make_double2(w * e.loss, w * e.kl);
  }
  __syncthreads();
  const RowGrad grad(told[1], told[0], static_cast<int>(label));
#pragma unroll
  for (int i = 0; i < R; ++i) {
    // widened anew: the registers hold the stored values alone in between
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    Words w = __builtin_bit_cast(Words, raw[i]);
    FINETUNE_OPAQUE(w);
    raw[i] = __builtin_bit_cast(typename Io::Vec, w);
    if (j + i * NT * V < p.last) store_vec<Io, STREAM>(o + j + i * NT * V, grad.piece<Io>(raw[i], j + i * NT * V));
  }
  if (column >= 0) {
    const float q = grad.at(extra);
    o[column] = Io::narrow(column == grad.label ? grad.g + q : q);
  }
}

}  // namespace finetune
