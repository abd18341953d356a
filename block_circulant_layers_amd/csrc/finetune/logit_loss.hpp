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
// r % positions).
template <class Io>
struct Rows {
  typename Io::T* data;
  int64_t seq_stride, pos_stride;
  __device__ __forceinline__ typename Io::T* row(int64_t r, int64_t positions) const {
    return data + (r / positions) * seq_stride + (r % positions) * pos_stride;
  }
};

// exp(d) for d <= 0 through the hardware's exp2.  log2(e) is taken as a sum of
// two floats: its rounding alone (1.3e-8) would shift every exponential, and
// with it every log-probability, the same way, which a sum over a sequence's
// positions does not average out.
__device__ __forceinline__ float exp_of(float d) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(d, 1.44269502162933349609375f, d * 1.925963033500011e-8f));
}

// A running maximum and the sum of exp(x - maximum).
struct MaxSum {
  float m = -INFINITY, s = 0.0f;
  __device__ __forceinline__ void add(float x) {
    if (x > m) {
      s = s * exp_of(m - x) + 1.0f;
      m = x;
    } else {
      s += x == m ? (m == -INFINITY ? 0.0f : 1.0f) : exp_of(x - m);
    }
  }
  __device__ __forceinline__ void join(float om, float os) {
    const float top = m > om ? m : om;
    if (top != m || top != om) {
      s = s * (m == top ? 1.0f : exp_of(m - top)) + os * (om == top ? 1.0f : exp_of(om - top));
      m = top;
    } else {
      s += os;
    }
  }
};

// lse and logp of every position, one workgroup per row.
template <class Io>
__global__ void __launch_bounds__(kLogitThreads)
    token_logprob_kernel(Rows<Io> in, const int64_t* labels, float* logp, float* lse, int64_t rows, int64_t positions,
                         int v) {
  __shared__ float sm[kLogitThreads / kWave], ss[kLogitThreads / kWave];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t label = labels[r];
    if (label < 0 || label >= v) {
      if (threadIdx.x == 0) logp[r] = lse[r] = label == kIgnore ? 0.0f : NAN;
      continue;
    }
    const typename Io::T* x = in.row(r, positions);
    MaxSum a;
    for (int j = threadIdx.x; j < v; j += kLogitThreads) a.add(Io::widen(x[j]));
#pragma unroll
    for (int o = kWave / 2; o > 0; o /= 2) a.join(__shfl_xor(a.m, o, kWave), __shfl_xor(a.s, o, kWave));
    if (threadIdx.x % kWave == 0) {
      sm[threadIdx.x / kWave] = a.m;
      ss[threadIdx.x / kWave] = a.s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < kLogitThreads / kWave; ++i) a.join(sm[i], ss[i]);
      // a.m - a.m: NaN for a row whose maximum is infinite (its softmax has no value)
      const double l = a.m + log(static_cast<double>(a.s)) + (a.m - a.m);
      lse[r] = static_cast<float>(l);
      logp[r] = static_cast<float>(Io::widen(x[label]) - l);
    }
    __syncthreads();
  }
}

// The gradient of every row: g = up[...] * slope[...], each either one value,
// one per sequence (modulo `up_n`), or one per position.
struct RowScale {
  const float* up;     // may be null (then `scale`)
  const float* slope;  // never null
  float scale;
  int64_t up_n;        // up is indexed by sequence modulo up_n
  bool slope_by_row;   // slope by row, else by sequence
  __device__ __forceinline__ float at(int64_t r, int64_t positions) const {
    const int64_t seq = r / positions;
    return (up ? up[seq % up_n] : scale) * slope[slope_by_row ? r : seq];
  }
};

template <class Io>
__global__ void __launch_bounds__(kLogitThreads)
    logits_grad_kernel(Rows<Io> in, const int64_t* labels, const float* lse, RowScale scale, Rows<Io> out,
                       int64_t rows, int64_t positions, int v) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int64_t label = labels[r];
    typename Io::T* o = out.row(r, positions);
    if (label == kIgnore) {
      for (int j = threadIdx.x; j < v; j += kLogitThreads) o[j] = Io::narrow(0.0f);
      continue;
    }
    const bool known = label >= 0 && label < v;
    const float g = known ? scale.at(r, positions) : NAN;
    const float l = lse[r];
    const typename Io::T* x = in.row(r, positions);
    for (int j = threadIdx.x; j < v; j += kLogitThreads) {
      const float p = exp_of(Io::widen(x[j]) - l);
      o[j] = Io::narrow(g * ((j == label ? 1.0f : 0.0f) - p));
    }
  }
}

struct Preference {
  int kind;
  bool average;
  double beta, smoothing;
};

// One workgroup per pair: both sequences' log-ratios, the loss and the slopes.
// The sums run in fp64 (a few values per thread).
__global__ void __launch_bounds__(kLogitThreads)
    preference_kernel(const int64_t* labels, const float* logp, const float* ref, Preference how, float* loss,
                      float* logratio, float* slope, int64_t pairs, int64_t positions) {
  __shared__ double s[2][kLogitThreads / kWave];
  __shared__ double n[2][kLogitThreads / kWave];
  for (int64_t b = blockIdx.x; b < pairs; b += gridDim.x) {
    double ratio[2], count[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int64_t base = (b + side * pairs) * positions;
      double a = 0.0, c = 0.0;
      for (int64_t i = threadIdx.x; i < positions; i += kLogitThreads)
        if (labels[base + i] != kIgnore) {
          a += static_cast<double>(logp[base + i]) - static_cast<double>(ref[base + i]);
          c += 1.0;
        }
      a = block_sum<kLogitThreads>(a, s[side]);
      c = block_sum<kLogitThreads>(c, n[side]);
      count[side] = how.average && c > 0.0 ? c : 1.0;
      ratio[side] = a / count[side];
    }
    if (threadIdx.x == 0) {
      const double h = ratio[0] - ratio[1], z = how.beta * h, e = how.smoothing;
      double l, dh;
      if (how.kind == 0) {
        const double t = log1p(exp(-fabs(z)));
        const double up = (z < 0.0 ? z : 0.0) - t;  // log sigma(z); log sigma(-z) = up - z
        l = -(1.0 - e) * up - e * (up - z);
        dh = -how.beta * ((1.0 - e) / (1.0 + exp(z)) - e / (1.0 + exp(-z)));
      } else if (how.kind == 1) {
        l = z < 1.0 ? 1.0 - z : z >= 1.0 ? 0.0 : z;  // the last: NaN
        dh = z < 1.0 ? -how.beta : z >= 1.0 ? 0.0 : z;
      } else {
        const double gap = h - 0.5 / how.beta;
        l = gap * gap;
        dh = 2.0 * gap;
      }
      loss[b] = static_cast<float>(l);
      logratio[b] = static_cast<float>(ratio[0]);
      logratio[b + pairs] = static_cast<float>(ratio[1]);
      slope[b] = static_cast<float>(dh / count[0]);
      slope[b + pairs] = static_cast<float>(-dh / count[1]);
    }
    __syncthreads();
  }
}

struct Policy {
  int reduction;
  bool per_token;
  double low, high, kl;
};

struct PolicyTerm {
  double loss, kl, slope;
};

// One position's loss, KL and d loss / d logp.
__device__ __forceinline__ PolicyTerm policy_term(const Policy& how, double logp, double old, const float* ref,
                                                  double adv) {
  PolicyTerm t{};
  const double r = exp(logp - old);
  const double lo = 1.0 - how.low, hi = 1.0 + how.high;
  const double held = (r < lo ? lo : r > hi ? hi : r) * adv, free = r * adv;
  t.loss = free > held ? -held : -free;  // a NaN ratio makes `free` NaN and stays
  t.slope = free > held ? 0.0 : -free;
  if (ref) {
    const double q = static_cast<double>(*ref) - logp, e = expm1(q);
    t.kl = e - q;
    t.loss += how.kl * t.kl;
    t.slope -= how.kl * e;
  }
  return t;
}

// Unmasked positions of every sequence, one workgroup per sequence.
__global__ void __launch_bounds__(kLogitThreads)
    count_kernel(const int64_t* labels, int* counts, int64_t seqs, int64_t positions) {
  __shared__ int s[kLogitThreads / kWave];
  for (int64_t q = blockIdx.x; q < seqs; q += gridDim.x) {
    int c = 0;
    for (int64_t i = threadIdx.x; i < positions; i += kLogitThreads) c += labels[q * positions + i] != kIgnore;
    c = block_sum<kLogitThreads>(c, s);
    if (threadIdx.x == 0) counts[q] = c;
    __syncthreads();
  }
}

// Every position's slope and the reduced loss and KL: one workgroup.
__global__ void __launch_bounds__(kLogitThreads)
    policy_kernel(const int64_t* labels, const float* logp, const float* old, const float* ref, const float* adv,
                  const int* counts, Policy how, float* stats, float* slope, int64_t seqs, int64_t positions) {
  __shared__ double s[3][kLogitThreads / kWave];
  double total = 0.0;
  for (int64_t q = threadIdx.x; q < seqs; q += kLogitThreads) total += counts[q];
  total = block_sum<kLogitThreads>(total, s[0]);
  double a = 0.0, k = 0.0;
  for (int64_t r = threadIdx.x; r < seqs * positions; r += kLogitThreads) {
    float out = 0.0f;
    if (labels[r] != kIgnore) {
      const int64_t q = r / positions;
      const double w = how.reduction == 0   ? 1.0 / total
                       : how.reduction == 1 ? 1.0 / (static_cast<double>(counts[q]) * static_cast<double>(seqs))
                                            : 1.0;
      const PolicyTerm t = policy_term(how, logp[r], old[r], ref ? ref + r : nullptr, adv[how.per_token ? r : q]);
      a += w * t.loss;
      k += w * t.kl;
      out = static_cast<float>(w * t.slope);
    }
    slope[r] = out;
  }
  a = block_sum<kLogitThreads>(a, s[1]);
  k = block_sum<kLogitThreads>(k, s[2]);
  if (threadIdx.x == 0) {
    stats[0] = static_cast<float>(a);
    stats[1] = static_cast<float>(k);
  }
}

}  // namespace finetune
