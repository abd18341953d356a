// attention_lib.hip -- C ABI of attention.h: argument checks, kernel selection, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attention.h"
#include "attention_launch.hpp"
#include "attention_validate.hpp"
#include "dropout.hpp"
#include "relative_bias.hpp"

namespace finetune {
namespace {

template <class F>
int by_dtype(int64_t dtype, F f) {
  switch (dtype) {
    case RDFFT_F32: return f(F32{});
    case RDFFT_BF16: return f(Bf16{});
    default: return f(F16{});
  }
}

// dtable[c, h] = the sum of its n partial sums, one wave each, in a fixed order
__global__ __launch_bounds__(kWave) void bias_parts_kernel(const float* part, float* dtable, int64_t n) {
  const float* mine = part + blockIdx.x * n;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kWave) s += mine[i];
  s = lanes_sum<kWave>(s);
  if (threadIdx.x == 0) dtable[blockIdx.x] = static_cast<float>(s);
}

constexpr int64_t kUnits = 256;  // compute units
// Buffers of a call beyond this many bytes go past the caches: they cannot be found there again.
constexpr int64_t kCacheBytes = int64_t(320) << 20;

// ---- relative position bias -----------------------------------------------

// The rule as the kernels take it.  A bucket's border falls on a whole distance where the two powers behind the
// logarithms are equal; the logarithm then misses the whole number by an ulp to either side, so what lies within
// 1e-9 of one counts as it (other distances of at most 1024 are further away).
Buckets buckets_of(const attention_buckets& b) {
  Buckets r{};
  r.count = static_cast<int>(b.count);
  r.two_sided = b.two_sided != 0;
  r.side = r.two_sided ? r.count / 2 : r.count;
  const int small = r.side / 2, rest = r.side - small;
  const double unit = std::log(static_cast<double>(b.max_distance) / small);
  for (int m = 0; m < small; ++m) r.first[m] = static_cast<int16_t>(m);
  int m = small;
  for (int n = small; m < r.side; ++n) {
    const int at = small + static_cast<int>(std::floor(std::log(static_cast<double>(n) / small) / unit * rest + 1e-9));
    for (; m < r.side && m <= at; ++m) r.first[m] = static_cast<int16_t>(n);
  }
  r.reach = r.first[r.side - 1];
  return r;
}

// row parts of a head: enough workgroups for the chip, no more than there is work for
int64_t bias_fwd_parts(int64_t heads, int64_t n) {
  return std::max<int64_t>(1, std::min(ceil_div(8 * kUnits, heads), ceil_div(n, 4 * kBiasThreads)));
}
int64_t bias_bwd_parts(int64_t heads, int64_t tq) {
  return std::max<int64_t>(1, std::min(ceil_div(8 * kUnits, heads), ceil_div(tq, 16)));
}

// ---- attention ------------------------------------------------------------

Problem problem_of(const attention_problem& a) {
  Problem p{};
  p.batch = static_cast<int>(a.batch), p.tq = static_cast<int>(a.queries), p.tk = static_cast<int>(a.keys);
  p.heads = static_cast<int>(a.heads), p.kv_heads = static_cast<int>(a.kv_heads);
  p.d = static_cast<int>(a.head_dim), p.group = p.heads / p.kv_heads, p.causal = a.causal != 0;
  p.scale = static_cast<float>(a.scale), p.scale2 = static_cast<float>(a.scale * 1.4426950408889634074);
  p.begin = a.key_begin, p.end = a.key_end, p.table = a.bias;
  return p;
}
// Heads of a group side by side in a workgroup's rows: for fewer queries than a workgroup has rows, where they
// share the loads of their key head (one query, 4096 keys, four heads to a key head: 17.3 us, 19.4 apart).  The bias
// differs from head to head.
int64_t pack_of(const attention_problem& a) {
  return !a.bias && a.queries < kAttnRows ? a.heads / a.kv_heads : 1;
}
// In how many parts a workgroup's walk over `steps` tiles is split: where workgroups fill at most half of the compute
// units, up to two a unit.  One query, 4096 keys, 8 key heads: 38 us in 32 parts of two tiles (29 of them the join, then
// one wave a row), 17.4 in 64 of one.  180 workgroups in two parts each: 16 us and 11 for the join, against 21.5 unsplit.
int64_t splits_of(int64_t blocks, int64_t steps) {
  if (blocks <= 0 || 2 * blocks > kUnits) return 1;
  return std::max<int64_t>(1, std::min(std::min(2 * kUnits / blocks, steps), int64_t(kMaxSplits)));
}

Plan plan_of(const attention_problem& a) {
  Plan p{};
  const int64_t rows = a.batch * a.heads * a.queries, keys = a.batch * a.kv_heads * a.keys, group = a.heads / a.kv_heads;
  p.pack = pack_of(a);
  const int64_t units = a.batch * a.kv_heads;
  p.fwd_blocks = units * (group / p.pack) * ceil_div(a.queries * p.pack, kAttnRows);
  p.fwd_splits = splits_of(p.fwd_blocks, ceil_div(a.keys, kAttnKeys));
  p.dq_blocks = units * group * ceil_div(a.queries, kAttnRows);
  p.q_splits = splits_of(p.dq_blocks, ceil_div(a.keys, kAttnKeys) / 2);
  const int64_t tiles = ceil_div(a.keys, kAttnRows);
  p.dkv_blocks = units * tiles;
  p.k_splits = splits_of(p.dkv_blocks, group * ceil_div(a.queries, kAttnKeys) / 2);
  const auto round4 = [](int64_t n) { return (n + 3) / 4 * 4; };
  if (p.fwd_splits > 1) p.fwd_bytes = 4 * (round4(p.fwd_splits * rows * a.head_dim) + round4(p.fwd_splits * rows * 2));
  int64_t at = 0;
  const auto take = [&](int64_t n) {
    const int64_t here = at;
    at += round4(n);
    return here;
  };
  p.delta = take(rows);
  p.peak = take(a.dtype == RDFFT_F16 ? rows : 0);
  p.dq = take(p.q_splits > 1 ? p.q_splits * rows * a.head_dim : 0);
  p.ddelta = take(p.q_splits > 1 ? p.q_splits * rows : 0);
  p.dk = take(p.k_splits > 1 ? p.k_splits * keys * a.head_dim : 0);
  p.dv = take(p.k_splits > 1 ? p.k_splits * keys * a.head_dim : 0);
  p.dbias = take(a.bias ? a.buckets.count * a.heads * a.batch * tiles * p.k_splits : 0);
  p.bwd_bytes = 4 * at;
  return p;
}
bool launchable(const attention_problem& a, const Plan& p) {
  return (!a.bias || a.buckets.count * a.heads <= kMaxBlocks) && p.fwd_blocks * p.fwd_splits <= kMaxBlocks && p.dq_blocks * p.q_splits <= kMaxBlocks &&
         p.dkv_blocks * p.k_splits <= kMaxBlocks;
}

}  // namespace
}  // namespace finetune

using namespace finetune;

extern "C" {

int attention_abi_version(void) { return ATTENTION_ABI_VERSION; }

int relative_bias_fwd(const float* table, void* bias, int64_t heads, int64_t queries, int64_t keys,
                      const attention_buckets* buckets, int dtype, void* stream) {
  const int st = check_bias_fwd(table, bias, heads, queries, keys, buckets, dtype);
  if (st != RDFFT_OK || queries == 0 || keys == 0) return st;
  const int64_t parts = bias_fwd_parts(heads, queries * keys);
  if (heads * parts > kMaxBlocks) return RDFFT_ERR_SIZE;
  const Buckets b = buckets_of(*buckets);
  return by_dtype(dtype, [&](auto io) {
    using Io = decltype(io);
    hipLaunchKernelGGL((relative_bias_fwd_kernel<Io>), dim3(static_cast<unsigned>(heads * parts)), dim3(kBiasThreads),
                       0, static_cast<hipStream_t>(stream), table, static_cast<typename Io::T*>(bias),
                       static_cast<int>(heads), queries, keys, static_cast<int>(parts), b);
    return launch_status();
  });
}

int relative_bias_workspace(int64_t batch, int64_t heads, int64_t queries, int64_t keys,
                            const attention_buckets* buckets, int64_t* bytes) {
  if (bytes == nullptr) return RDFFT_ERR_NULL;
  const int st = check_buckets(buckets);
  if (st != RDFFT_OK) return st;
  if (!valid_dims(batch, heads, queries, keys)) return RDFFT_ERR_SIZE;
  const bool none = batch == 0 || queries == 0 || keys == 0;
  *bytes = none ? 0 : ceil_div(buckets->count * heads * bias_bwd_parts(heads, queries) * 4, 16) * 16;
  return RDFFT_OK;
}

int relative_bias_bwd(const void* dbias, int64_t batch_stride, int64_t head_stride, int64_t query_stride,
                      float* dtable, int64_t batch, int64_t heads, int64_t queries, int64_t keys,
                      const attention_buckets* buckets, void* ws, int64_t ws_bytes, int dtype, void* stream) {
  int64_t need = 0;
  int st = relative_bias_workspace(batch, heads, queries, keys, buckets, &need);
  if (st != RDFFT_OK && valid_dtype(dtype)) return st;
  const int64_t stride[3] = {batch_stride, head_stride, query_stride};
  st = check_bias_bwd(dbias, stride, dtable, batch, heads, queries, keys, buckets, ws, ws_bytes, need, dtype);
  if (st != RDFFT_OK) return st;
  const bool none = batch == 0 || queries == 0 || keys == 0;
  const int64_t parts = none ? 0 : bias_bwd_parts(heads, queries);
  if (heads * parts > kMaxBlocks || buckets->count * heads > kMaxBlocks) return RDFFT_ERR_SIZE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!none) {
    const Buckets b = buckets_of(*buckets);
    st = by_dtype(dtype, [&](auto io) {
      using Io = decltype(io);
      const int lds = 4 * kBiasThreads / kWave * Slots(b.reach + Io::kVec).size();
      const dim3 grid(static_cast<unsigned>(heads * parts));
      const auto* from = static_cast<const typename Io::T*>(dbias);
      auto* to = static_cast<float*>(ws);
      if (batch * heads * queries * keys * int64_t(sizeof(typename Io::T)) > kCacheBytes)
        hipLaunchKernelGGL((relative_bias_bwd_kernel<Io, true>), grid, dim3(kBiasThreads), lds, s, from, batch_stride,
                           head_stride, query_stride, to, batch, queries, keys, static_cast<int>(parts), b);
      else
        hipLaunchKernelGGL((relative_bias_bwd_kernel<Io, false>), grid, dim3(kBiasThreads), lds, s, from, batch_stride,
                           head_stride, query_stride, to, batch, queries, keys, static_cast<int>(parts), b);
      return launch_status();
    });
    if (st != RDFFT_OK) return st;
  }
  hipLaunchKernelGGL((bias_parts_kernel), dim3(static_cast<unsigned>(buckets->count * heads)), dim3(kWave), 0, s,
                     static_cast<const float*>(ws), dtable, parts);
  return launch_status();
}

int attention_workspace(const attention_problem* a, int backward, int64_t* bytes) {
  if (bytes == nullptr) return RDFFT_ERR_NULL;
  const int st = check_problem(a);
  if (st != RDFFT_OK) return st;
  const Plan p = plan_of(*a);
  if (!launchable(*a, p)) return RDFFT_ERR_SIZE;
  *bytes = backward ? p.bwd_bytes : p.fwd_bytes;
  return RDFFT_OK;
}

int attention_fwd(const attention_problem* a, const attention_tensor* q, const attention_tensor* k,
                  const attention_tensor* v, const attention_tensor* o, float* lse, void* ws, int64_t ws_bytes,
                  void* stream) {
  int64_t need = 0;
  int st = attention_workspace(a, 0, &need);
  if (st != RDFFT_OK) return st;
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr) return RDFFT_ERR_NULL;
  Rows4 in[3] = {rows4(*a, *q, false), rows4(*a, *k, true), rows4(*a, *v, true)}, out = rows4(*a, *o, false);
  for (Rows4& r : in)
    if ((st = check_tensor(r, false)) != RDFFT_OK) return st;
  if ((st = check_tensor(out, true)) != RDFFT_OK) return st;
  if (out.empty()) return RDFFT_OK;
  if (lse == nullptr) return RDFFT_ERR_NULL;
  if (!aligned_to(lse, 4)) return RDFFT_ERR_ALIGN;
  if ((st = check_workspace(ws, ws_bytes, need)) != RDFFT_OK) return st;
  const Range small[] = {{lse, a->batch * a->heads * a->queries * 4}, {ws, need}};
  const Range read[] = {{a->key_begin, a->batch * 4}, {a->key_end, a->batch * 4},
                        {a->bias, a->bias ? a->buckets.count * a->heads * 4 : 0}};
  for (const Rows4& r : in)
    if (clash(out, r)) return RDFFT_ERR_ALIAS;
  for (const Range& w : small) {
    for (const Rows4& r : in)
      if (clash(r, w.p, w.bytes)) return RDFFT_ERR_ALIAS;
    if (clash(out, w.p, w.bytes) || clashes(w, read)) return RDFFT_ERR_ALIAS;
  }
  for (const Range& r : read)
    if (clash(out, r.p, r.bytes)) return RDFFT_ERR_ALIAS;
  if (clashes(small[0], small[1])) return RDFFT_ERR_ALIAS;

  const Plan plan = plan_of(*a);
  const Problem p = problem_of(*a);
  const Buckets b = a->bias ? buckets_of(a->buckets) : Buckets{};
  const int64_t rows = a->batch * a->heads * a->queries;
  FwdParts parts{static_cast<float*>(ws), nullptr, static_cast<int>(plan.fwd_splits)};
  parts.stats = parts.o + ceil_div(plan.fwd_splits * rows * a->head_dim, 4) * 4;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const FwdCall call{p, plan, view_of(*q), view_of(*k), view_of(*v), view_of(*o), lse, parts, b, s};
  return by_dtype(a->dtype, [&](auto io) { return launch_fwd<decltype(io)>(call); });
}

int attention_bwd(const attention_problem* a, const attention_tensor* q, const attention_tensor* k,
                  const attention_tensor* v, const attention_tensor* o, const float* lse,
                  const attention_tensor* dout, const attention_tensor* dq, const attention_tensor* dk,
                  const attention_tensor* dv, float* dbias, void* ws, int64_t ws_bytes, void* stream) {
  int64_t need = 0;
  int st = attention_workspace(a, 1, &need);
  if (st != RDFFT_OK) return st;
  if (!q || !k || !v || !o || !dout || !dq || !dk || !dv) return RDFFT_ERR_NULL;
  if (dbias && !a->bias) return RDFFT_ERR_SHAPE;
  Rows4 in[5] = {rows4(*a, *q, false), rows4(*a, *k, true), rows4(*a, *v, true), rows4(*a, *o, false),
                 rows4(*a, *dout, false)};
  Rows4 out[3] = {rows4(*a, *dq, false), rows4(*a, *dk, true), rows4(*a, *dv, true)};
  for (Rows4& r : in)
    if ((st = check_tensor(r, false)) != RDFFT_OK) return st;
  for (Rows4& r : out)
    if ((st = check_tensor(r, true)) != RDFFT_OK) return st;
  const int64_t rows = a->batch * a->heads * a->queries;
  if (rows > 0 && lse == nullptr) return RDFFT_ERR_NULL;
  if (!aligned_to(lse, 4) || !aligned_to(dbias, 4)) return RDFFT_ERR_ALIGN;
  if ((st = check_workspace(ws, ws_bytes, need)) != RDFFT_OK) return st;
  const int64_t table = a->bias ? a->buckets.count * a->heads * 4 : 0;
  const Range small[] = {{dbias, table}, {ws, need}};
  const Range read[] = {{lse, rows * 4}, {a->key_begin, a->batch * 4}, {a->key_end, a->batch * 4}, {a->bias, table}};
  for (int n = 0; n < 3; ++n) {
    for (const Rows4& r : in)
      if (clash(out[n], r)) return RDFFT_ERR_ALIAS;
    for (int m = n + 1; m < 3; ++m)
      if (clash(out[n], out[m])) return RDFFT_ERR_ALIAS;
    for (const Range& r : read)
      if (clash(out[n], r.p, r.bytes)) return RDFFT_ERR_ALIAS;
    for (const Range& w : small)
      if (clash(out[n], w.p, w.bytes)) return RDFFT_ERR_ALIAS;
  }
  for (const Range& w : small) {
    for (const Rows4& r : in)
      if (clash(r, w.p, w.bytes)) return RDFFT_ERR_ALIAS;
    if (clashes(w, read)) return RDFFT_ERR_ALIAS;
  }
  if (clashes(small[0], small[1])) return RDFFT_ERR_ALIAS;

  const Plan plan = plan_of(*a);
  const Problem p = problem_of(*a);
  const Buckets b = a->bias ? buckets_of(a->buckets) : Buckets{};
  float* w = static_cast<float*>(ws);
  const BwdParts parts{w + plan.delta, w + plan.peak, w + plan.dq, w + plan.ddelta, w + plan.dk, w + plan.dv,
                       dbias ? w + plan.dbias : nullptr, static_cast<int>(plan.q_splits),
                       static_cast<int>(plan.k_splits)};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const BwdCall call{p,  plan, view_of(*q), view_of(*k), view_of(*v), view_of(*o), view_of(*dout), view_of(*dq),
                     view_of(*dk), view_of(*dv), lse, parts, b, s};
  st = by_dtype(a->dtype, [&](auto io) { return launch_bwd<decltype(io)>(call); });
  if (st != RDFFT_OK || dbias == nullptr) return st;
  const int64_t n = plan.dkv_blocks > 0 ? a->batch * ceil_div(a->keys, kAttnRows) * plan.k_splits : 0;
  hipLaunchKernelGGL((bias_parts_kernel), dim3(static_cast<unsigned>(a->buckets.count * a->heads)), dim3(kWave), 0, s,
                     w + plan.dbias, dbias, n);
  return launch_status();
}

}  // extern "C"

namespace finetune {
namespace {

template <bool RES>
int launch_dropout(const void* x, const void* res, void* y, const DropArgs& a, int dtype, hipStream_t s) {
  return by_dtype(dtype, [&](auto io) {
    using Io = decltype(io);
    using T = typename Io::T;
    const auto *px = static_cast<const T*>(x), *pr = static_cast<const T*>(res);
    auto* py = static_cast<T*>(y);
    const int64_t n = a.rows * a.d;
    const int64_t grid = std::min(ceil_div(n / 8 + 1, kDropThreads), 8 * kUnits);
    const bool flat = a.rows == 1 || (a.xs == a.d && a.ys == a.d && (!RES || a.rs == a.d));
    if (!flat) {
      hipLaunchKernelGGL((dropout_rows_kernel<Io, RES>), dim3(static_cast<unsigned>(grid)), dim3(kDropThreads), 0, s,
                         px, pr, py, a);
    } else if (n * int64_t(sizeof(T)) * (RES ? 3 : 2) > kCacheBytes) {
      hipLaunchKernelGGL((dropout_kernel<Io, RES, true>), dim3(static_cast<unsigned>(grid)), dim3(kDropThreads), 0, s,
                         px, pr, py, n, a);
    } else {
      hipLaunchKernelGGL((dropout_kernel<Io, RES, false>), dim3(static_cast<unsigned>(grid)), dim3(kDropThreads), 0,
                         s, px, pr, py, n, a);
    }
    return launch_status();
  });
}

DropArgs drop_args(int64_t rows, int64_t d, int64_t xs, int64_t rs, int64_t ys, const attention_dropout& how) {
  const double least = std::nearbyint(how.p * 65536.0);
  return {rows, d, xs, rs, ys, how.seed, how.offset, how.device_seed, static_cast<uint32_t>(least),
          least < 65536.0 ? static_cast<float>(65536.0 / (65536.0 - least)) : 0.0f};
}

}  // namespace
}  // namespace finetune

extern "C" {

int dropout_fwd(const void* x, const void* residual, void* y, int64_t rows, int64_t d, int64_t x_stride,
                int64_t residual_stride, int64_t y_stride, const attention_dropout* how, int dtype, void* stream) {
  const int st = check_dropout(x, residual, y, rows, d, x_stride, residual_stride, y_stride, how, dtype);
  if (st != RDFFT_OK || rows == 0) return st;
  const DropArgs a = drop_args(rows, d, x_stride, residual_stride, y_stride, *how);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return residual ? launch_dropout<true>(x, residual, y, a, dtype, s) : launch_dropout<false>(x, nullptr, y, a, dtype, s);
}

int dropout_bwd(const void* dy, void* dx, int64_t rows, int64_t d, int64_t dy_stride, int64_t dx_stride,
                const attention_dropout* how, int dtype, void* stream) {
  const int st = check_dropout(dy, nullptr, dx, rows, d, dy_stride, 0, dx_stride, how, dtype);
  if (st != RDFFT_OK || rows == 0) return st;
  return launch_dropout<false>(dy, nullptr, dx, drop_args(rows, d, dy_stride, 0, dx_stride, *how), dtype,
                               static_cast<hipStream_t>(stream));
}

}  // extern "C"
