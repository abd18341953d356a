// finetune_lib.hip -- C ABI of libfinetune.so: argument checks, kernel selection, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "finetune.h"
#include "grad_clip.hpp"
#include "layer_norm.hpp"
#include "logit_loss.hpp"
#include "validate.hpp"

namespace finetune {
namespace {

int launch_status() { return hipGetLastError() == hipSuccess ? RDFFT_OK : RDFFT_ERR_LAUNCH; }

template <class F>
int by_dtype(int64_t dtype, F f) {
  switch (dtype) {
    case RDFFT_F32: return f(F32{});
    case RDFFT_BF16: return f(Bf16{});
    default: return f(F16{});
  }
}

template <class T>
struct TypeOf {
  using type = T;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether a call's large buffers of `bytes` in all go past the caches: where the
// 256 MB cache cannot hold them until they are used again.  Both sides, layer
// norm of rows of 4096 bf16: forward of 16384 rows (268 MB) 52 us past the
// caches, 48 through them, of 32768 rows 101 and 107; backward of 8192 rows
// (201 MB) 43 and 43, of 16384 rows (403 MB) 76 and 79.
// (This size and the numbers of workgroups below are smaller in a host build
// that runs the kernels on CPU threads.)
#ifndef FINETUNE_CACHE_BYTES
#define FINETUNE_CACHE_BYTES (int64_t(320) << 20)
#endif
constexpr bool past_caches(int64_t bytes) { return bytes > FINETUNE_CACHE_BYTES; }
template <class F>
void by_stream(bool stream, F f) {
  if (stream)
    f(std::true_type{});
  else
    f(std::false_type{});
}

constexpr int64_t kMaxGrid = 1 << 20;
unsigned grid_of(int64_t n) { return static_cast<unsigned>(n < kMaxGrid ? n : kMaxGrid); }

// ---- layer normalisation --------------------------------------------------

// threads that hold a row of d elements, 0 for the kernels of any length
int norm_threads(int64_t d) {
  for (int t = 8; t <= 1024; t *= 2)
    if (d <= t * kNormElems) return t;
  return 0;
}

// f(std::integral_constant<int, T>, std::bool_constant<RAGGED>) for a row of d elements of Io
template <class Io, class F>
void by_norm_row(int64_t d, F f) {
  auto ragged = [&](auto t) {
    if (d % Io::kVec)
      f(t, std::true_type{});
    else
      f(t, std::false_type{});
  };
  switch (norm_threads(d)) {
    case 8: ragged(std::integral_constant<int, 8>{}); break;
    case 16: ragged(std::integral_constant<int, 16>{}); break;
    case 32: ragged(std::integral_constant<int, 32>{}); break;
    case 64: ragged(std::integral_constant<int, 64>{}); break;
    case 128: ragged(std::integral_constant<int, 128>{}); break;
    case 256: ragged(std::integral_constant<int, 256>{}); break;
    case 512: ragged(std::integral_constant<int, 512>{}); break;
    default: ragged(std::integral_constant<int, 1024>{}); break;
  }
}

// Workgroups of the backward, each with one slice of the sums over rows (the
// kernels of any length: row ranges of the column kernel).  One a compute unit
// keeps enough loads in flight, and every other one makes slices to write and
// sum: rows of 4096 bf16, 256 / 512 / 1024 workgroups: 2048 rows 20 / 25 / 36 us,
// 16384 rows 80 / 86 / 102 us.  Rows of up to 1024 elements have slices small
// enough for two a unit (32768 rows of 512: 30 / 25.5 / 27 us).
#ifndef FINETUNE_NORM_GROUPS
#define FINETUNE_NORM_GROUPS 256  // one a compute unit
#endif
constexpr int64_t kNormGroups = FINETUNE_NORM_GROUPS;
struct DwSplit {
  int64_t parts, per;
};
DwSplit dw_split(int64_t rows, int64_t d) {
  const int t = norm_threads(d);
  if (t) {
    const int64_t groups = ceil_div(std::max<int64_t>(rows, 1), norm_wg(t) / t);
    return {std::min<int64_t>(groups, t >= kNormThreads ? kNormGroups : 2 * kNormGroups), 0};
  }
  const int64_t cols = ceil_div(d, kNormThreads);
  const int64_t parts = std::max<int64_t>(std::min<int64_t>(1024 / cols, ceil_div(rows, 16)), 1);
  const int64_t per = std::max<int64_t>(ceil_div(rows, parts), 1);
  return {std::max<int64_t>(ceil_div(rows, per), 1), per};
}

template <class Io>
int launch_norm_fwd(const void* x, const float* w, const float* b, void* y, float* mean, float* rstd, int64_t rows,
                    int64_t d, int64_t xs, int64_t ys, double eps, hipStream_t s) {
  using T = typename Io::T;
  const auto* px = static_cast<const T*>(x);
  auto* py = static_cast<T*>(y);
  const int n = static_cast<int>(d);
  if (norm_threads(d) == 0) {
    hipLaunchKernelGGL((layer_norm_wide_fwd_kernel<Io>), dim3(grid_of(rows)), dim3(kNormThreads), 0, s, px, w, b, py,
                       mean, rstd, rows, n, xs, ys, static_cast<float>(eps));
    return launch_status();
  }
  by_norm_row<Io>(d, [&](auto t, auto ragged) {
    constexpr int TT = decltype(t)::value, WG = norm_wg(TT);
    const int64_t groups = ceil_div(rows, WG / TT);
    const int64_t grid = std::min<int64_t>(groups, 8 * kNormGroups * kNormThreads / WG);  // 32 waves a compute unit
    by_stream(past_caches(2 * rows * d * int64_t(sizeof(T))), [&](auto stream) {
      hipLaunchKernelGGL((layer_norm_fwd_kernel<Io, TT, decltype(ragged)::value, decltype(stream)::value>),
                         dim3(static_cast<unsigned>(grid)), dim3(WG), 0, s, px, w, b, py, mean, rstd, rows, n, xs, ys,
                         static_cast<float>(eps));
    });
  });
  return launch_status();
}

template <class Io>
int launch_norm_bwd(const void* x, const float* w, const float* mean, const float* rstd, const void* dy, void* dx,
                    float* ws, const DwSplit& split, int64_t rows, int64_t d, int64_t xs, int64_t dys, int64_t dxs,
                    hipStream_t s) {
  using T = typename Io::T;
  const auto *px = static_cast<const T*>(x), *pg = static_cast<const T*>(dy);
  auto* po = static_cast<T*>(dx);
  const int n = static_cast<int>(d);
  if (norm_threads(d)) {
    by_norm_row<Io>(d, [&](auto t, auto ragged) {
      constexpr int TT = decltype(t)::value;
      by_stream(past_caches(3 * rows * d * int64_t(sizeof(T))), [&](auto stream) {
        hipLaunchKernelGGL((layer_norm_bwd_kernel<Io, TT, decltype(ragged)::value, decltype(stream)::value>),
                           dim3(static_cast<unsigned>(split.parts)), dim3(norm_wg(TT)), norm_bwd_lds(TT), s, px, w,
                           mean, rstd, pg, po, ws, rows, n, xs, dys, dxs);
      });
    });
    return launch_status();
  }
  if (ws) {  // the sums first: dx may replace the dy they read
    hipLaunchKernelGGL((layer_norm_wide_dw_kernel<Io>),
                       dim3(static_cast<unsigned>(ceil_div(d, kNormThreads)), static_cast<unsigned>(split.parts)),
                       dim3(kNormThreads), 0, s, px, mean, rstd, pg, ws, rows, n, xs, dys, split.per);
    const int st = launch_status();
    if (st != RDFFT_OK) return st;
  }
  if (po)
    hipLaunchKernelGGL((layer_norm_wide_dx_kernel<Io>), dim3(grid_of(rows)), dim3(kNormThreads), 0, s, px, w, mean,
                       rstd, pg, po, rows, n, xs, dys, dxs);
  return launch_status();
}

// ---- logits ---------------------------------------------------------------

template <class Io>
Rows<Io> rows_of(const finetune_logits* in) {
  return {static_cast<typename Io::T*>(const_cast<void*>(in->data)), in->seq_stride, in->pos_stride};
}
template <class Io>
Rows<Io> rows_of(const finetune_dlogits* out) {
  return {static_cast<typename Io::T*>(out->data), out->seq_stride, out->pos_stride};
}

// How a launch over rows of `vocab` columns is split: `nt` threads a
// workgroup, `parts` workgroups of `per` columns a row.  A row of up to four
// pieces a lane takes one wave, of up to 16 where kManyRows fill the chip with
// waves: no barrier, and one reduction of lanes.  (One wave a row / a workgroup a
// row, bf16, a forward and a step: 16384 rows of 2000, 24 / 35 us and 43 / 61 us;
// of 8000, 45 / 56 and 104 / 112; 4096 of 8000, 19.4 / 19.9 and 38.8 / 37.9; 1024
// of 8000, 13.1 / 12.5 and 22.0 / 20.7.  16384 rows of 16000: 65 / 72 and 199 /
// 197.)  Fewer rows than kWantGroups workgroups, two a
// compute unit, are split until there are as many, or until a part holds one
// piece a thread.  (With 1024 as the limit, 999 rows of 10007 fp32 took 15.1 us
// in two parts each and their joins, 13.4 us whole; a step of 512 rows of 50001
// bf16 31 us in parts, 27 us with the rows held.)
#ifndef FINETUNE_WANT_GROUPS
#define FINETUNE_WANT_GROUPS 512
#endif
constexpr int64_t kWantGroups = FINETUNE_WANT_GROUPS;
constexpr int64_t kManyRows = 8 * kWantGroups;
struct RowSplit {
  int nt, parts, per;
};
RowSplit row_split(const finetune_logits* in) {
  const int64_t v = in->vocab, piece = in->dtype == RDFFT_F32 ? 4 : 8;
  const int64_t rows = logit_rows(in), lane = rows < kManyRows ? 4 : 16;  // pieces a lane of a row's one wave
  RowSplit s{v <= lane * kWave * piece ? kWave : kLogitThreads, 1, static_cast<int>(v)};
  if (rows > 0 && rows < kWantGroups && s.nt == kLogitThreads) {
    const int64_t unit = s.nt * piece;
    const int64_t parts = std::min<int64_t>(ceil_div(kWantGroups, rows), ceil_div(v, unit));
    const int64_t per = ceil_div(ceil_div(v, parts), unit) * unit;
    s.parts = static_cast<int>(ceil_div(v, per));
    s.per = static_cast<int>(per);
  }
  return s;
}

template <class F>
void by_threads(int nt, F f) {
  if (nt == kWave)
    f(std::integral_constant<int, kWave>{});
  else
    f(std::integral_constant<int, kLogitThreads>{});
}

// Workspace of the calls on logits: one total, a count a sequence, two fp64
// shares a row (policy loss), and the parts of split rows (a maximum and a sum
// each) with their labels' logits.
struct LogitsWorkspace {
  int64_t counts, terms, parts, picked, bytes;  // offsets, and the size
  explicit LogitsWorkspace(const finetune_logits* in) {
    const auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
    const RowSplit s = row_split(in);
    counts = 16;
    terms = counts + up(in->seqs * 4);
    parts = terms + logit_rows(in) * 16;
    picked = parts + (s.parts > 1 ? up(logit_rows(in) * s.parts * 8) : 0);
    bytes = picked + (s.parts > 1 ? up(logit_rows(in) * 4) : 0);
  }
};
int64_t logits_workspace(const finetune_logits* in) { return LogitsWorkspace(in).bytes; }
template <class T>
T* at(void* ws, int64_t offset) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + offset);
}

template <class Io>
JoinParts<Io> join_of(const finetune_logits* in, const RowSplit& split, float* lse, void* ws) {
  int lanes = 1;
  while (lanes < split.parts && lanes < kWave) lanes *= 2;
  return {rows_of<Io>(in), split.parts > 1 ? at<const float2>(ws, LogitsWorkspace(in).parts) : nullptr,
          at<const float>(ws, LogitsWorkspace(in).picked), lse, split.parts, lanes, static_cast<int>(in->vocab)};
}

int64_t logit_bytes(const finetune_logits* in) {
  return logit_rows(in) * in->vocab * dtype_bytes(static_cast<int>(in->dtype));
}

// Logits at the end of a batch that a step reads through the caches, because
// their gradient reads them again and starts there: the size of the cache and
// what masked rows, which are not read, leave of it.  4 x 1024 pairs of 50001
// bf16, none / 100 / 200 / 256 / 320 / 400 / 512 MB / all of them: 366 / 358 / 352
// / 344 / 341 / 340 / 340 / 347 us; 8 x 512 of 32768: 215 us with none, 190 us
// with 400 MB.
constexpr int64_t kKeepBytes = int64_t(400) << 20;

// the rows' log-probabilities, or, where rows are split, their parts; `again`:
// a gradient follows
template <class Io>
int launch_rows(const finetune_logits* in, const RowSplit& split, float* logp, float* lse, bool again, void* ws,
                hipStream_t s) {
  const int64_t rows = logit_rows(in);
  if (rows == 0) return RDFFT_OK;
  const int64_t keep = again ? std::max<int64_t>(rows - kKeepBytes / ceil_div(logit_bytes(in), rows), 0) : rows;
  by_threads(split.nt, [&](auto nt) {
    by_stream(past_caches(logit_bytes(in)), [&](auto stream) {
      constexpr int NT = decltype(nt)::value;
      hipLaunchKernelGGL((token_logprob_kernel<Io, NT, decltype(stream)::value>), dim3(grid_of(rows * split.parts)),
                         dim3(NT), 0, s, rows_of<Io>(in), in->labels, logp, lse,
                         at<float2>(ws, LogitsWorkspace(in).parts), at<float>(ws, LogitsWorkspace(in).picked), rows,
                         in->positions,
                         static_cast<int>(in->vocab), split.parts, split.per, keep);
    });
  });
  return launch_status();
}

int launch_logprob(const finetune_logits* in, float* logp, float* lse, void* ws, hipStream_t s) {
  return by_dtype(in->dtype, [&](auto io) {
    using Io = decltype(io);
    const RowSplit split = row_split(in);
    const int st = launch_rows<Io>(in, split, logp, lse, false, ws, s);
    if (st != RDFFT_OK || split.parts == 1) return st;
    const int64_t rows = logit_rows(in);
    hipLaunchKernelGGL((join_kernel<Io>), dim3(static_cast<unsigned>(ceil_div(rows, kJoinRows))), dim3(kLogitThreads),
                       0, s, join_of<Io>(in, split, lse, ws), in->labels, logp, rows);
    return launch_status();
  });
}

int launch_grad(const finetune_logits* in, const float* lse, const RowScale& scale, const finetune_dlogits* out,
                hipStream_t s) {
  const int64_t rows = logit_rows(in);
  if (rows == 0) return RDFFT_OK;
  return by_dtype(in->dtype, [&](auto io) {
    using Io = decltype(io);
    const RowSplit split = row_split(in);
    by_threads(split.nt, [&](auto nt) {
      by_stream(past_caches(2 * logit_bytes(in)), [&](auto stream) {
        constexpr int NT = decltype(nt)::value;
        hipLaunchKernelGGL((logits_grad_kernel<Io, NT, decltype(stream)::value>), dim3(grid_of(rows * split.parts)),
                           dim3(NT), 0, s, rows_of<Io>(in), in->labels, lse, scale, rows_of<Io>(out), rows,
                           in->positions, static_cast<int>(in->vocab), split.parts, split.per);
      });
    });
    return launch_status();
  });
}

Preference preference_of(const finetune_preference* how) {
  return {static_cast<int>(how->kind), how->average != 0, how->beta, how->smoothing};
}

int launch_preference(const finetune_logits* in, const float* ref, const finetune_preference* how,
                      const PreferenceOut& res, float* logp, float* lse, bool again, void* ws, hipStream_t s) {
  if (in->seqs == 0) return RDFFT_OK;
  const int64_t pairs = in->seqs / 2;
  return by_dtype(in->dtype, [&](auto io) {
    using Io = decltype(io);
    const RowSplit split = row_split(in);
    const int st = launch_rows<Io>(in, split, logp, lse, again, ws, s);
    if (st != RDFFT_OK) return st;
    hipLaunchKernelGGL((preference_kernel<Io>), dim3(grid_of(pairs)), dim3(kPairThreads), 0, s,
                       join_of<Io>(in, split, lse, ws), in->labels, logp, ref, preference_of(how), res, pairs,
                       in->positions);
    return launch_status();
  });
}

// Whether a step's gradient kernel works the slopes out for itself: rows enough
// to fill the chip would each repeat what one launch does once.
bool few_rows(const finetune_logits* in) { return logit_rows(in) > 0 && logit_rows(in) < kWantGroups; }
// ... with `more` workgroups for what is not a row's gradient
unsigned few_rows_grid(const finetune_logits* in, const RowSplit& split, int64_t more) {
  return static_cast<unsigned>(more + logit_rows(in) * split.parts);
}

int launch_preference_step(const finetune_logits* in, const float* ref, const finetune_preference* how, float scale,
                           const PreferenceOut& res, float* logp, float* lse, const finetune_dlogits* out, void* ws,
                           hipStream_t s) {
  if (!few_rows(in)) {
    const int st = launch_preference(in, ref, how, res, logp, lse, true, ws, s);
    if (st != RDFFT_OK) return st;
    return launch_grad(in, lse, RowScale{nullptr, res.slope, scale, 1, false}, out, s);
  }
  return by_dtype(in->dtype, [&](auto io) {
    using Io = decltype(io);
    const RowSplit split = row_split(in);
    const int st = launch_rows<Io>(in, split, logp, lse, true, ws, s);
    if (st != RDFFT_OK) return st;
    hipLaunchKernelGGL((preference_grad_kernel<Io>), dim3(few_rows_grid(in, split, in->seqs / 2)),
                       dim3(kLogitThreads), 0, s, join_of<Io>(in, split, lse, ws), in->labels, logp, ref, preference_of(how), scale, res,
                       rows_of<Io>(out), in->seqs / 2, in->positions, split.parts, split.per);
    return launch_status();
  });
}

// Rows up to which one workgroup does all that follows the log-probabilities
// (8192 rows took one workgroup 32 us, three launches 13 us).
constexpr int64_t kPolicyOne = 2048;
static_assert(kPolicyOne >= kWantGroups, "rows in parts are joined by that workgroup");

// what policy kernels share
struct PolicyCall {
  Policy how;
  PolicyInputs in;
  PolicyWeight weight;
  int *counts, *total;
  double2* terms;
};
PolicyCall policy_call(const finetune_logits* in, const float* old, const float* ref, const float* adv,
                       const finetune_policy* how, void* ws) {
  const LogitsWorkspace w(in);
  const int reduction = static_cast<int>(how->reduction);
  int *counts = at<int>(ws, w.counts), *total = at<int>(ws, 0);
  return {{reduction, how->clip_low, how->clip_high, how->kl_coef},
          {old, ref, adv, how->advantage_per_token != 0},
          {counts, total, reduction, in->seqs},
          counts,
          total,
          at<double2>(ws, w.terms)};
}

int launch_policy_count(const finetune_logits* in, const PolicyCall& c, hipStream_t s) {
  if (c.how.reduction == POLICY_SUM) return RDFFT_OK;
  hipLaunchKernelGGL((policy_count_kernel), dim3(1), dim3(kPolicyThreads), 0, s, in->labels, c.counts, c.total,
                     c.how.reduction, in->seqs, in->positions);
  return launch_status();
}

int launch_policy_sum(const finetune_logits* in, const PolicyCall& c, float* stats, hipStream_t s) {
  hipLaunchKernelGGL((policy_sum_kernel), dim3(1), dim3(kPolicyThreads), 0, s, c.terms, stats, logit_rows(in));
  return launch_status();
}

int launch_policy(const finetune_logits* in, const PolicyCall& c, float* stats, float* logp, float* lse, float* slope,
                  bool again, void* ws, hipStream_t s) {
  return by_dtype(in->dtype, [&](auto io) {
    using Io = decltype(io);
    const RowSplit split = row_split(in);
    const int64_t rows = logit_rows(in);
    int st = launch_rows<Io>(in, split, logp, lse, again, ws, s);
    if (st != RDFFT_OK) return st;
    if (rows <= kPolicyOne) {
      hipLaunchKernelGGL((policy_kernel<Io>), dim3(1), dim3(kPolicyThreads), 0, s, join_of<Io>(in, split, lse, ws),
                         in->labels, logp, c.in, c.weight, c.counts, c.total, c.how, stats, slope, in->seqs,
                         in->positions);
      return launch_status();
    }
    st = launch_policy_count(in, c, s);
    if (st != RDFFT_OK) return st;
    hipLaunchKernelGGL((policy_rows_kernel), dim3(grid_of(ceil_div(rows, kLogitThreads))), dim3(kLogitThreads), 0, s,
                       in->labels, logp, c.in, c.weight, c.how, slope, c.terms, rows, in->positions);
    st = launch_status();
    return st == RDFFT_OK ? launch_policy_sum(in, c, stats, s) : st;
  });
}

// The step with the rows held in registers, where there are rows enough to fill
// the chip and a row fits a workgroup: f(threads, pieces a thread), and whether
// there was such a shape.  A workgroup takes one row (it has no registers to
// spare for a loop's), and HIP launches fewer than 2^32 threads: batches past
// that take the kernels that walk over the rows.
constexpr int64_t kLaunchThreads = (int64_t(1) << 32) - 1;
template <class F>
bool by_held_row(const finetune_logits* in, F f) {
  const int64_t pieces = in->vocab / (in->dtype == RDFFT_F32 ? 4 : 8);
  const auto with = [&](auto nt, auto r) {
    if (logit_rows(in) > kLaunchThreads / decltype(nt)::value) return false;
    f(nt, r);
    return true;
  };
  if (logit_rows(in) < kWantGroups) return false;
  if (pieces <= 64 * 8) return with(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
  if (pieces <= 256 * 8) return with(std::integral_constant<int, 256>{}, std::integral_constant<int, 8>{});
  if (pieces <= 512 * 16) return with(std::integral_constant<int, 512>{}, std::integral_constant<int, 16>{});
  if (pieces <= 1024 * 16) return with(std::integral_constant<int, 1024>{}, std::integral_constant<int, 16>{});
  return false;
}

int launch_policy_step(const finetune_logits* in, const PolicyCall& c, float scale, float* stats, float* logp,
                       float* lse, float* slope, const finetune_dlogits* out, void* ws, hipStream_t s) {
  if (few_rows(in))
    return by_dtype(in->dtype, [&](auto io) {
      using Io = decltype(io);
      const RowSplit split = row_split(in);
      const int st = launch_rows<Io>(in, split, logp, lse, true, ws, s);
      if (st != RDFFT_OK) return st;
      hipLaunchKernelGGL((policy_grad_kernel<Io>), dim3(few_rows_grid(in, split, 1)), dim3(kLogitThreads), 0, s,
                         join_of<Io>(in, split, lse, ws), in->labels, logp, c.in, c.weight, c.counts, c.total, c.how,
                         scale, stats, slope, rows_of<Io>(out), in->seqs, in->positions, split.parts, split.per);
      return launch_status();
    });
  const bool held = by_held_row(in, [](auto, auto) {});
  if (!held) {
    const int st = launch_policy(in, c, stats, logp, lse, slope, true, ws, s);
    if (st != RDFFT_OK) return st;
    return launch_grad(in, lse, RowScale{nullptr, slope, scale, 1, true}, out, s);
  }
  int st = launch_policy_count(in, c, s);
  if (st != RDFFT_OK) return st;
  st = by_dtype(in->dtype, [&](auto io) {
    using Io = decltype(io);
    by_held_row(in, [&](auto nt, auto r) {
      by_stream(past_caches(2 * logit_bytes(in)), [&](auto stream) {
        constexpr int NT = decltype(nt)::value, R = decltype(r)::value;
        hipLaunchKernelGGL((policy_step_kernel<Io, NT, R, decltype(stream)::value>),
                           dim3(static_cast<unsigned>(logit_rows(in))), dim3(NT), 0, s, rows_of<Io>(in), in->labels,
                           c.in, c.weight, c.how, scale, logp, lse, slope, c.terms, rows_of<Io>(out), in->positions,
                           static_cast<int>(in->vocab));
      });
    });
    return launch_status();
  });
  return st == RDFFT_OK ? launch_policy_sum(in, c, stats, s) : st;
}

// ---- gradient tensors -----------------------------------------------------

// f(table, chunks) for tables of up to Table::kMost tensors, the chunks of a
// launch below 2^24, laid out along the lines of the tensors read (BACK:
// written); BACK: the last tensor first.
template <class Table, bool BACK, class F>
int for_tables(const finetune_tensor* t, int64_t n, F f) {
  constexpr int64_t kMost = int64_t(1) << 23, kEntryChunks = int64_t(1) << 16;
  static_assert(kEntryChunks * kClipBytes / 2 < kClipEntry, "an entry's elements fit its count");
  Table table;
  table.n = 0;
  table.first[0] = 0;
  auto flush = [&]() {
    if (table.n == 0) return static_cast<int>(RDFFT_OK);
    const int st = f(table, table.first[table.n]);
    table.n = 0;
    return st;
  };
  for (int64_t at = 0; at < n; ++at) {
    const finetune_tensor& x = t[BACK ? n - 1 - at : at];
    int64_t left = x.count;
    const int size = static_cast<int>(dtype_bytes(static_cast<int>(x.dtype)));
    const int64_t per = kClipBytes / size;
    const char* g = static_cast<const char*>(x.grad);
    char* o = static_cast<char*>(x.out);
    while (left > 0) {
      const int64_t take = std::min<int64_t>(left, kEntryChunks * per);
      const int64_t chunks = ceil_div(take + clip_lead(BACK ? o : g, size), per);
      const int k = table.n++;
      table.in[k] = g;
      if constexpr (Table::kApart) table.to[k] = o;
      table.count[k] = static_cast<uint32_t>(x.dtype) * kClipEntry + static_cast<uint32_t>(take);
      table.first[k + 1] = table.first[k] + static_cast<int>(chunks);
      left -= take;
      g += take * size;
      if (o) o += take * size;
      if (table.n == Table::kMost || table.first[table.n] >= kMost) {
        const int st = flush();
        if (st != RDFFT_OK) return st;
      }
    }
  }
  return flush();
}

unsigned clip_grid(int chunks) { return static_cast<unsigned>(std::min(chunks, kClipGroups)); }

// partial sums and chunks of all launches of squares
struct ClipShape {
  int64_t parts = 0, chunks = 0;
  ClipShape(const finetune_tensor* t, int64_t n) {
    for_tables<ClipHere, false>(t, n, [&](const ClipHere&, int c) {
      parts += clip_grid(c);
      chunks += c;
      return static_cast<int>(RDFFT_OK);
    });
  }
  int64_t workspace() const { return (parts * 8 + 15) / 16 * 16; }
};

// The chunks at the end that the squares read through the caches, because the
// scaling starts there.  50 tensors of 537 MB, none / 128 / 256 / 400 MB / all of
// it: 275 / 270 / 260 / 264 / 266 us; 200 tensors of 805 MB: 427 us with none, 416
// with 256 MB.
constexpr int64_t kClipKeepChunks = (int64_t(256) << 20) / kClipBytes;

int launch_squares(const finetune_tensor* t, int64_t n, const ClipShape& shape, bool again, double* partial,
                   hipStream_t s) {
  int64_t keep = shape.chunks * kClipBytes * (again ? 2 : 1);
  keep = !past_caches(keep) ? 0 : again ? shape.chunks - kClipKeepChunks : shape.chunks;
  return for_tables<ClipHere, false>(t, n, [&](const ClipHere& table, int chunks) {
    const int here = static_cast<int>(std::max<int64_t>(std::min<int64_t>(keep, chunks), 0));
    hipLaunchKernelGGL((grad_square_kernel), dim3(clip_grid(chunks)), dim3(kClipThreads), 0, s, table, here, partial);
    partial += clip_grid(chunks);
    keep -= chunks;
    return launch_status();
  });
}

int launch_norm(const double* partial, int64_t parts, float* norm, hipStream_t s) {
  hipLaunchKernelGGL((grad_norm_kernel), dim3(1), dim3(kClipThreads), 0, s, partial, parts, norm);
  return launch_status();
}

// the launches over the tables, the first of them with the norm's address
int launch_scale(const finetune_tensor* t, int64_t n, const ClipShape& shape, const double* partial, double max_norm,
                 double eps, float* norm, hipStream_t s) {
  const auto over = [&](auto kind) {
    using Table = typename decltype(kind)::type;
    return for_tables<Table, true>(t, n, [&](const Table& table, int chunks) {
      by_stream(past_caches(2 * shape.chunks * kClipBytes), [&](auto stream) {
        hipLaunchKernelGGL((grad_scale_kernel<Table, decltype(stream)::value>), dim3(clip_grid(chunks)),
                           dim3(kClipThreads), 0, s, table, partial, shape.parts, max_norm, eps, norm);
      });
      norm = nullptr;
      return launch_status();
    });
  };
  const auto apart = [](const finetune_tensor& x) { return x.count > 0 && x.out != x.grad; };
  return std::any_of(t, t + n, apart) ? over(TypeOf<ClipApart>{}) : over(TypeOf<ClipHere>{});
}

}  // namespace
}  // namespace finetune

using namespace finetune;

extern "C" {

int finetune_abi_version(void) { return FINETUNE_ABI_VERSION; }

const char* finetune_status_string(int status) {
  switch (status) {
    case RDFFT_OK: return "ok";
    case RDFFT_ERR_NULL: return "null pointer";
    case RDFFT_ERR_SIZE: return "a count or parameter outside its range, or a workspace too small";
    case RDFFT_ERR_SHAPE: return "strides or counts that do not go together";
    case RDFFT_ERR_DTYPE: return "unsupported dtype";
    case RDFFT_ERR_ALIGN: return "a pointer without its element's alignment";
    case RDFFT_ERR_ALIAS: return "output buffer overlaps another buffer";
    case RDFFT_ERR_LAUNCH: return "kernel launch failed";
    default: return "unknown status";
  }
}

int layer_norm_fwd(const void* x, const float* weight, const float* bias, void* y, float* mean, float* rstd,
                   int64_t rows, int64_t d, int64_t x_stride, int64_t y_stride, double eps, int dtype, void* stream) {
  const int st = check_norm_fwd(x, weight, bias, y, mean, rstd, rows, d, x_stride, y_stride, eps, dtype);
  if (st != RDFFT_OK || rows == 0) return st;
  return by_dtype(dtype, [&](auto io) {
    return launch_norm_fwd<decltype(io)>(x, weight, bias, y, mean, rstd, rows, d, x_stride, y_stride, eps,
                                         static_cast<hipStream_t>(stream));
  });
}

int layer_norm_bwd_workspace(int64_t rows, int64_t d, int64_t* bytes) {
  if (bytes == nullptr) return RDFFT_ERR_NULL;
  const int st = check_norm_dims(rows, d);
  if (st == RDFFT_OK) *bytes = rows == 0 ? 0 : (dw_split(rows, d).parts * 2 * d * 4 + 15) / 16 * 16;
  return st;
}

int layer_norm_bwd(const void* x, const float* weight, const float* mean, const float* rstd, const void* dy, void* dx,
                   float* dweight, float* dbias, void* ws, int64_t ws_bytes, int64_t rows, int64_t d,
                   int64_t x_stride, int64_t dy_stride, int64_t dx_stride, int dtype, void* stream) {
  int64_t need = 0;
  int st = layer_norm_bwd_workspace(rows, d, &need);
  if (st == RDFFT_OK || !valid_dtype(dtype))
    st = check_norm_bwd(x, weight, mean, rstd, dy, dx, dweight, dbias, ws, ws_bytes, need, rows, d, x_stride,
                        dy_stride, dx_stride, dtype);
  if (st != RDFFT_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const DwSplit split = dw_split(rows, d);
  const bool sums = dweight || dbias;
  if (rows > 0) {
    st = by_dtype(dtype, [&](auto io) {
      return launch_norm_bwd<decltype(io)>(x, weight, mean, rstd, dy, dx, sums ? static_cast<float*>(ws) : nullptr,
                                           split, rows, d, x_stride, dy_stride, dx_stride, s);
    });
    if (st != RDFFT_OK) return st;
  }
  if (!sums) return RDFFT_OK;
  hipLaunchKernelGGL((layer_norm_dw_sum_kernel), dim3(static_cast<unsigned>(ceil_div(2 * d, kSumCols))),
                     dim3(kSumCols * kSumGroups), 0, s, static_cast<const float*>(ws), dweight, dbias,
                     static_cast<int>(d), rows > 0 ? static_cast<int>(split.parts) : 0);
  return launch_status();
}

int finetune_logits_workspace(const finetune_logits* in, int64_t* bytes) {
  if (bytes == nullptr) return RDFFT_ERR_NULL;
  const int st = check_logits_dims(in);
  if (st == RDFFT_OK) *bytes = logits_workspace(in);
  return st;
}

int token_logprob(const finetune_logits* in, float* logp, float* lse, void* ws, int64_t ws_bytes, void* stream) {
  int st = check_logits(in);
  if (st != RDFFT_OK) return st;
  const int64_t rows = logit_rows(in), need = logits_workspace(in);
  st = check_workspace(ws, ws_bytes, need);
  const Array none[] = {{nullptr, 0}}, outs[] = {{logp, rows}, {lse, rows}};
  if (st == RDFFT_OK) st = check_arrays(in, nullptr, none, outs, ws, need);
  if (st != RDFFT_OK) return st;
  return launch_logprob(in, logp, lse, ws, static_cast<hipStream_t>(stream));
}

int token_logprob_bwd(const finetune_logits* in, const float* lse, const float* dlogp, const finetune_dlogits* out,
                      void* stream) {
  int st = check_logits(in);
  if (st == RDFFT_OK) st = check_dlogits(in, out);
  if (st != RDFFT_OK) return st;
  const int64_t rows = logit_rows(in);
  const Array ins[] = {{lse, rows}, {dlogp, rows}}, none[] = {{nullptr, 0}};
  st = check_arrays(in, out, ins, none, nullptr, 0);
  if (st != RDFFT_OK) return st;
  return launch_grad(in, lse, RowScale{nullptr, dlogp, 1.0f, 1, true}, out, static_cast<hipStream_t>(stream));
}

int preference_loss_fwd(const finetune_logits* in, const float* ref_logp, const finetune_preference* how, float* loss,
                        float* logratio, float* logp, float* lse, float* slope, void* ws, int64_t ws_bytes,
                        void* stream) {
  int st = check_logits(in);
  if (st == RDFFT_OK) st = check_preference(in, how);
  if (st != RDFFT_OK) return st;
  const int64_t rows = logit_rows(in), need = logits_workspace(in);
  st = check_workspace(ws, ws_bytes, need);
  const Array ins[] = {{ref_logp, rows}};
  const Array outs[] = {{loss, in->seqs / 2}, {logratio, in->seqs}, {logp, rows}, {lse, rows}, {slope, in->seqs}};
  if (st == RDFFT_OK) st = check_arrays(in, nullptr, ins, outs, ws, need);
  if (st != RDFFT_OK) return st;
  return launch_preference(in, ref_logp, how, PreferenceOut{loss, logratio, slope}, logp, lse, false, ws,
                           static_cast<hipStream_t>(stream));
}

int preference_loss_bwd(const finetune_logits* in, const float* lse, const float* slope, const float* dloss,
                        const finetune_dlogits* out, void* stream) {
  int st = check_logits(in);
  if (st == RDFFT_OK && in->seqs % 2 != 0) st = RDFFT_ERR_SHAPE;
  if (st == RDFFT_OK) st = check_dlogits(in, out);
  if (st != RDFFT_OK) return st;
  const Array ins[] = {{lse, logit_rows(in)}, {slope, in->seqs}, {dloss, in->seqs / 2}}, none[] = {{nullptr, 0}};
  st = check_arrays(in, out, ins, none, nullptr, 0);
  if (st != RDFFT_OK) return st;
  return launch_grad(in, lse, RowScale{dloss, slope, 1.0f, in->seqs / 2, false}, out,
                     static_cast<hipStream_t>(stream));
}

int preference_loss_step(const finetune_logits* in, const float* ref_logp, const finetune_preference* how,
                         double scale, float* loss, float* logratio, float* logp, float* lse, float* slope,
                         const finetune_dlogits* out, void* ws, int64_t ws_bytes, void* stream) {
  int st = check_logits(in);
  if (st == RDFFT_OK) st = check_preference(in, how);
  if (st == RDFFT_OK) st = check_dlogits(in, out);
  if (st != RDFFT_OK) return st;
  const int64_t rows = logit_rows(in), need = logits_workspace(in);
  st = check_workspace(ws, ws_bytes, need);
  const Array ins[] = {{ref_logp, rows}};
  const Array outs[] = {{loss, in->seqs / 2}, {logratio, in->seqs}, {logp, rows}, {lse, rows}, {slope, in->seqs}};
  if (st == RDFFT_OK) st = check_arrays(in, out, ins, outs, ws, need);
  if (st != RDFFT_OK) return st;
  return launch_preference_step(in, ref_logp, how, static_cast<float>(scale), PreferenceOut{loss, logratio, slope},
                                logp, lse, out, ws, static_cast<hipStream_t>(stream));
}

int policy_loss_fwd(const finetune_logits* in, const float* old_logp, const float* ref_logp, const float* advantages,
                    const finetune_policy* how, float* stats, float* logp, float* lse, float* slope, void* ws,
                    int64_t ws_bytes, void* stream) {
  int st = check_logits(in);
  if (st == RDFFT_OK) st = check_policy(how);
  if (st != RDFFT_OK) return st;
  const int64_t rows = logit_rows(in), need = logits_workspace(in);
  st = check_workspace(ws, ws_bytes, need);
  const Array ins[] = {{old_logp, rows}, {ref_logp, rows, true}, {advantages, how->advantage_per_token ? rows : in->seqs}};
  const Array outs[] = {{stats, 2}, {logp, rows}, {lse, rows}, {slope, rows}};
  if (st == RDFFT_OK) st = check_arrays(in, nullptr, ins, outs, ws, need);
  if (st != RDFFT_OK) return st;
  return launch_policy(in, policy_call(in, old_logp, ref_logp, advantages, how, ws), stats, logp, lse, slope, false,
                       ws, static_cast<hipStream_t>(stream));
}

int policy_loss_bwd(const finetune_logits* in, const float* lse, const float* slope, const float* dloss,
                    const finetune_dlogits* out, void* stream) {
  int st = check_logits(in);
  if (st == RDFFT_OK) st = check_dlogits(in, out);
  if (st != RDFFT_OK) return st;
  const int64_t rows = logit_rows(in);
  const Array ins[] = {{lse, rows}, {slope, rows}, {dloss, 1}}, none[] = {{nullptr, 0}};
  st = check_arrays(in, out, ins, none, nullptr, 0);
  if (st != RDFFT_OK) return st;
  return launch_grad(in, lse, RowScale{dloss, slope, 1.0f, 1, true}, out, static_cast<hipStream_t>(stream));
}

int policy_loss_step(const finetune_logits* in, const float* old_logp, const float* ref_logp, const float* advantages,
                     const finetune_policy* how, double scale, float* stats, float* logp, float* lse, float* slope,
                     const finetune_dlogits* out, void* ws, int64_t ws_bytes, void* stream) {
  int st = check_logits(in);
  if (st == RDFFT_OK) st = check_policy(how);
  if (st == RDFFT_OK) st = check_dlogits(in, out);
  if (st != RDFFT_OK) return st;
  const int64_t rows = logit_rows(in), need = logits_workspace(in);
  st = check_workspace(ws, ws_bytes, need);
  const Array ins[] = {{old_logp, rows}, {ref_logp, rows, true}, {advantages, how->advantage_per_token ? rows : in->seqs}};
  const Array outs[] = {{stats, 2}, {logp, rows}, {lse, rows}, {slope, rows}};
  if (st == RDFFT_OK) st = check_arrays(in, out, ins, outs, ws, need);
  if (st != RDFFT_OK) return st;
  return launch_policy_step(in, policy_call(in, old_logp, ref_logp, advantages, how, ws), static_cast<float>(scale),
                            stats, logp, lse, slope, out, ws, static_cast<hipStream_t>(stream));
}

int grad_norm_workspace(const finetune_tensor* tensors, int64_t n, int64_t* bytes) {
  if (bytes == nullptr) return RDFFT_ERR_NULL;
  if (n < 0 || n > kMaxTensors) return RDFFT_ERR_SIZE;
  if (n > 0 && tensors == nullptr) return RDFFT_ERR_NULL;
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i)
    if (tensors[i].count < 0 || tensors[i].count > kMaxElems || (total += tensors[i].count) > kMaxElems)
      return RDFFT_ERR_SIZE;
  *bytes = ClipShape(tensors, n).workspace();
  return RDFFT_OK;
}

int grad_norm(const finetune_tensor* tensors, int64_t n, float* norm, void* ws, int64_t ws_bytes, void* stream) {
  int st = check_tensors(tensors, n, false);
  if (st != RDFFT_OK) return st;
  const ClipShape shape(tensors, n);
  st = check_norm_buffers(tensors, n, false, norm, ws, ws_bytes, shape.workspace());
  if (st != RDFFT_OK) return st;
  auto* partial = static_cast<double*>(ws);
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = launch_squares(tensors, n, shape, false, partial, s);
  return st == RDFFT_OK ? launch_norm(partial, shape.parts, norm, s) : st;
}

int clip_grad_norm(const finetune_tensor* tensors, int64_t n, double max_norm, double eps, float* norm, void* ws,
                   int64_t ws_bytes, void* stream) {
  int st = check_tensors(tensors, n, true);
  if (st == RDFFT_OK && (!(max_norm >= 0.0) || !(eps >= 0.0))) st = RDFFT_ERR_SIZE;
  if (st != RDFFT_OK) return st;
  const ClipShape shape(tensors, n);
  st = check_norm_buffers(tensors, n, true, norm, ws, ws_bytes, shape.workspace());
  if (st == RDFFT_OK) st = check_tensor_aliases(tensors, n);
  if (st != RDFFT_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto* partial = static_cast<double*>(ws);
  st = launch_squares(tensors, n, shape, true, partial, s);
  if (st != RDFFT_OK) return st;
  if (shape.parts == 0) return launch_norm(partial, 0, norm, s);  // no elements at all
  return launch_scale(tensors, n, shape, partial, max_norm, eps, norm, s);
}

}  // extern "C"
