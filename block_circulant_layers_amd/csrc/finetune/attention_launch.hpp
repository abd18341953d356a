// attention_launch.hpp -- the launches of the attention kernels, one storage type a source file
// (attention_f32.hip, attention_bf16.hip, attention_f16.hip instantiate them).
#pragma once

#include <type_traits>

#include "attention.h"
#include "attention_bwd.hpp"
#include "attention_fwd.hpp"

namespace finetune {

inline int launch_status() { return hipGetLastError() == hipSuccess ? RDFFT_OK : RDFFT_ERR_LAUNCH; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline View view_of(const attention_tensor& t) { return {t.data, t.batch_stride, t.token_stride, t.head_stride}; }


// What a call's work is cut into, and its workspace.
struct Plan {
  int64_t pack, fwd_blocks, fwd_splits;
  int64_t dq_blocks, q_splits, dkv_blocks, k_splits;
  int64_t fwd_bytes, bwd_bytes;
  // offsets of the backward's workspace, in floats
  int64_t delta, peak, dq, ddelta, dk, dv, dbias;
};

struct FwdCall {
  Problem a;
  Plan plan;
  View q, k, v, o;
  float* lse;
  FwdParts parts;
  Buckets buckets;
  hipStream_t s;
};
struct BwdCall {
  Problem a;
  Plan plan;
  View q, k, v, o, dout, dq, dk, dv;
  const float* lse;
  BwdParts parts;
  Buckets buckets;
  hipStream_t s;
};

// f(std::integral_constant<int, DP>) with the padded head size
template <class F>
int by_head(int64_t d, F f) {
  if (d <= 32) return f(std::integral_constant<int, 32>{});
  if (d <= 64) return f(std::integral_constant<int, 64>{});
  if (d <= 96) return f(std::integral_constant<int, 96>{});
  return f(std::integral_constant<int, 128>{});
}
template <class F>
int by_bias(bool bias, F f) {
  return bias ? f(std::true_type{}) : f(std::false_type{});
}

template <class Io>
int launch_fwd(const FwdCall& c) {
  const int64_t blocks = c.plan.fwd_blocks * c.plan.fwd_splits, rows = int64_t(c.a.batch) * c.a.heads * c.a.tq;
  const int code = by_head(c.a.d, [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    return by_bias(c.a.table, [&](auto bias) {
      constexpr bool kBias = decltype(bias)::value;
      const int lds = 2 * Tile<Io, DP>::bytes(kAttnKeys) + (kBias ? 4 * bias_line(c.buckets) : 0);
      hipLaunchKernelGGL((attention_fwd_kernel<Io, DP, kBias>), dim3(static_cast<unsigned>(blocks)),
                         dim3(kAttnThreads), lds, c.s, c.a, c.q, c.k, c.v, c.o, c.lse, c.parts,
                         static_cast<int>(c.plan.pack), c.buckets);
      return launch_status();
    });
  });
  if (code != RDFFT_OK || c.plan.fwd_splits == 1) return code;
  const dim3 grid(static_cast<unsigned>(rows));
  if (c.plan.fwd_splits > 8)
    hipLaunchKernelGGL((attention_join_kernel<Io, 8>), grid, dim3(8 * kWave), 0, c.s, c.a, c.o, c.lse, c.parts);
  else
    hipLaunchKernelGGL((attention_join_kernel<Io, 1>), grid, dim3(kWave), 0, c.s, c.a, c.o, c.lse, c.parts);
  return launch_status();
}

template <class Io>
int launch_bwd(const BwdCall& c) {
  const Problem& a = c.a;
  const int64_t rows = int64_t(a.batch) * a.heads * a.tq, keys = int64_t(a.batch) * a.kv_heads * a.tk;
  return by_head(a.d, [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    return by_bias(a.table, [&](auto bias) {
      constexpr bool kBias = decltype(bias)::value;
      const int line = kBias ? 4 * bias_line(c.buckets) : 0;
      const int dq_lds = 2 * Tile<Io, DP>::bytes(kAttnKeys) + line;
      const int dkv_lds = 2 * 4 * kTileSet<Io, DP> +
                          (kBias ? line + 4 * 4 * (kBlockFloats + Slots(c.buckets.reach + kEdge).size()) : 0);
      int code = RDFFT_OK;
      if (c.plan.dq_blocks > 0) {
        hipLaunchKernelGGL((attention_dq_kernel<Io, DP, kBias>),
                           dim3(static_cast<unsigned>(c.plan.dq_blocks * c.plan.q_splits)), dim3(kAttnThreads),
                           dq_lds, c.s, a, c.q, c.k, c.v, c.o, c.dout, c.lse, c.dq, c.parts, c.buckets);
        code = launch_status();
        if (code == RDFFT_OK && c.plan.q_splits > 1) {
          hipLaunchKernelGGL((attention_sum_kernel<Io>), dim3(static_cast<unsigned>(rows)), dim3(kWave), 0, c.s,
                             SumJob{c.parts.dq, c.dq}, SumJob{}, c.parts.q_splits, rows, a.heads, a.tq, a.d,
                             c.parts.ddelta, c.parts.delta);
          code = launch_status();
        }
      }
      if (code != RDFFT_OK || c.plan.dkv_blocks == 0) return code;
      hipLaunchKernelGGL((attention_dkv_kernel<Io, DP, kBias>),
                         dim3(static_cast<unsigned>(c.plan.dkv_blocks * c.plan.k_splits)),
                         dim3(kAttnThreads), dkv_lds, c.s, a, c.q, c.k, c.v, c.dout, c.lse, c.dk, c.dv, c.parts, c.buckets);
      code = launch_status();
      if (code != RDFFT_OK || c.plan.k_splits == 1) return code;
      hipLaunchKernelGGL((attention_sum_kernel<Io>), dim3(static_cast<unsigned>(2 * keys)), dim3(kWave), 0, c.s,
                         SumJob{c.parts.dk, c.dk}, SumJob{c.parts.dv, c.dv}, c.parts.k_splits, keys, a.kv_heads, a.tk,
                         a.d, static_cast<const float*>(nullptr), static_cast<float*>(nullptr));
      return launch_status();
    });
  });
}

extern template int launch_fwd<F32>(const FwdCall&);
extern template int launch_fwd<Bf16>(const FwdCall&);
extern template int launch_fwd<F16>(const FwdCall&);
extern template int launch_bwd<F32>(const BwdCall&);
extern template int launch_bwd<Bf16>(const BwdCall&);
extern template int launch_bwd<F16>(const BwdCall&);

}  // namespace finetune
