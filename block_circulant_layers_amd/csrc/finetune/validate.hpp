// validate.hpp -- host-side argument checks of finetune.h (no HIP calls).
//
// Every entry point runs these before enqueuing anything; on failure it
// returns the status and touches no device memory.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "finetune.h"
#include "../rdfft_validate.hpp"

namespace finetune {

using rdfft::aligned16;
using rdfft::dtype_bytes;
using rdfft::kMaxElems;
using rdfft::overlaps;
using rdfft::valid_dtype;

constexpr int64_t kMaxWidth = int64_t(1) << 20;   // of a normalised row
constexpr int64_t kMaxVocab = int64_t(1) << 24;   // of a row of logits
constexpr int64_t kMaxTensors = int64_t(1) << 20;

inline bool aligned_to(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

inline int check_workspace(const void* ws, int64_t ws_bytes, int64_t need) {
  if (ws_bytes < need || ws_bytes < 0) return RDFFT_ERR_SIZE;
  if (need == 0) return RDFFT_OK;
  if (ws == nullptr) return RDFFT_ERR_NULL;
  return aligned16(ws) ? RDFFT_OK : RDFFT_ERR_ALIGN;
}

// ---- layer normalisation --------------------------------------------------

inline int check_norm_dims(int64_t rows, int64_t d) {
  if (d < 1 || d > kMaxWidth || rows < 0 || rows > 0x7fffffff || rows > kMaxElems / d) return RDFFT_ERR_SIZE;
  return RDFFT_OK;
}

// rows of d elements `stride` apart, within the element limit
inline bool valid_rows(int64_t rows, int64_t d, int64_t stride) {
  return stride >= d && (rows <= 1 || stride <= kMaxElems / rows);
}
inline int64_t span(int64_t rows, int64_t d, int64_t stride) { return rows > 0 ? (rows - 1) * stride + d : 0; }

struct Range {
  const void* p;
  int64_t bytes;
};
inline bool clashes(const Range& a, const Range& b) { return overlaps(a.p, a.bytes, b.p, b.bytes); }
template <size_t N>
inline bool clashes(const Range& a, const Range (&others)[N]) {
  for (const Range& b : others)
    if (clashes(a, b)) return true;
  return false;
}

inline int check_norm_fwd(const void* x, const float* w, const float* b, const void* y, const float* mean,
                          const float* rstd, int64_t rows, int64_t d, int64_t xs, int64_t ys, double eps, int dtype) {
  if (!valid_dtype(dtype)) return RDFFT_ERR_DTYPE;
  if (check_norm_dims(rows, d) != RDFFT_OK || !(eps >= 0.0) || isinf(eps)) return RDFFT_ERR_SIZE;
  if (rows == 0) return RDFFT_OK;
  if (!valid_rows(rows, d, xs) || !valid_rows(rows, d, ys)) return RDFFT_ERR_SHAPE;
  if (x == nullptr || y == nullptr) return RDFFT_ERR_NULL;
  const int64_t e = dtype_bytes(dtype);
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(w, 4) || !aligned_to(b, 4) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return RDFFT_ERR_ALIGN;
  const Range in[] = {{w, d * 4}, {b, d * 4}}, rx{x, span(rows, d, xs) * e}, ry{y, span(rows, d, ys) * e},
              rm{mean, rows * 4}, rr{rstd, rows * 4};
  if (!(x == y && xs == ys) && clashes(ry, rx)) return RDFFT_ERR_ALIAS;
  if (clashes(ry, in) || clashes(rm, in) || clashes(rr, in) || clashes(rm, rx) || clashes(rr, rx) ||
      clashes(rm, ry) || clashes(rr, ry) || clashes(rm, rr))
    return RDFFT_ERR_ALIAS;
  return RDFFT_OK;
}

inline int check_norm_bwd(const void* x, const float* w, const float* mean, const float* rstd, const void* dy,
                          const void* dx, const float* dw, const float* db, const void* ws, int64_t ws_bytes,
                          int64_t need, int64_t rows, int64_t d, int64_t xs, int64_t dys, int64_t dxs, int dtype) {
  if (!valid_dtype(dtype)) return RDFFT_ERR_DTYPE;
  if (check_norm_dims(rows, d) != RDFFT_OK) return RDFFT_ERR_SIZE;
  if (dx == nullptr && dw == nullptr && db == nullptr) return RDFFT_ERR_NULL;
  if (!aligned_to(dw, 4) || !aligned_to(db, 4)) return RDFFT_ERR_ALIGN;
  if (overlaps(dw, d * 4, db, d * 4)) return RDFFT_ERR_ALIAS;
  if (rows == 0) return RDFFT_OK;
  if (!valid_rows(rows, d, xs) || !valid_rows(rows, d, dys) || (dx && !valid_rows(rows, d, dxs)))
    return RDFFT_ERR_SHAPE;
  if (x == nullptr || mean == nullptr || rstd == nullptr || dy == nullptr) return RDFFT_ERR_NULL;
  const int64_t e = dtype_bytes(dtype);
  if (!aligned_to(x, e) || !aligned_to(dy, e) || !aligned_to(dx, e) || !aligned_to(w, 4) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return RDFFT_ERR_ALIGN;
  if (dw || db) {
    const int st = check_workspace(ws, ws_bytes, need);
    if (st != RDFFT_OK) return st;
  } else {
    need = 0;
  }
  const Range in[] = {{x, span(rows, d, xs) * e}, {w, d * 4}, {mean, rows * 4}, {rstd, rows * 4}};
  const Range rdy{dy, span(rows, d, dys) * e}, rdx{dx, dx ? span(rows, d, dxs) * e : 0}, rdw{dw, d * 4},
      rdb{db, d * 4}, rws{ws, need};
  if (!(dx == dy && dxs == dys) && clashes(rdx, rdy)) return RDFFT_ERR_ALIAS;
  const Range written[] = {rdx, rdw, rdb, rws};
  for (const Range& o : written)
    if (clashes(o, in)) return RDFFT_ERR_ALIAS;
  if (clashes(rdw, rdy) || clashes(rdb, rdy) || clashes(rws, rdy) || clashes(rdx, rdw) || clashes(rdx, rdb) ||
      clashes(rdx, rws) || clashes(rdw, rws) || clashes(rdb, rws))
    return RDFFT_ERR_ALIAS;
  return RDFFT_OK;
}

// ---- logits ---------------------------------------------------------------

inline int check_logits_dims(const finetune_logits* in) {
  if (in == nullptr) return RDFFT_ERR_NULL;
  if (in->dtype < 0 || in->dtype > 2) return RDFFT_ERR_DTYPE;
  if (in->seqs < 0 || in->positions < 0 || in->vocab < 1 || in->vocab > kMaxVocab || in->seqs > 0x7fffffff ||
      in->positions > 0x7fffffff || in->seqs * in->positions > 0x7fffffff)
    return RDFFT_ERR_SIZE;
  return RDFFT_OK;
}

inline int64_t logit_rows(const finetune_logits* in) { return in->seqs * in->positions; }

// elements from the first to one past the last of a strided [seqs, positions, vocab]
inline int64_t logit_span(const finetune_logits* in, int64_t ss, int64_t ps) {
  return logit_rows(in) > 0 ? (in->seqs - 1) * ss + (in->positions - 1) * ps + in->vocab : 0;
}
inline bool valid_strides(const finetune_logits* in, int64_t ss, int64_t ps) {
  return ss >= 0 && ps >= 0 && (in->seqs <= 1 || ss <= kMaxElems / in->seqs) &&
         (in->positions <= 1 || ps <= kMaxElems / in->positions);
}

inline int check_logits(const finetune_logits* in) {
  const int st = check_logits_dims(in);
  if (st != RDFFT_OK) return st;
  if (logit_rows(in) == 0) return RDFFT_OK;
  if (!valid_strides(in, in->seq_stride, in->pos_stride)) return RDFFT_ERR_SHAPE;
  if (in->data == nullptr || in->labels == nullptr) return RDFFT_ERR_NULL;
  if (!aligned_to(in->data, dtype_bytes(int(in->dtype))) || !aligned_to(in->labels, 8)) return RDFFT_ERR_ALIGN;
  return RDFFT_OK;
}

inline Range range_of(const finetune_logits* in) {
  return {in->data, logit_span(in, in->seq_stride, in->pos_stride) * dtype_bytes(int(in->dtype))};
}
inline Range range_of_labels(const finetune_logits* in) { return {in->labels, logit_rows(in) * 8}; }

// the gradient's buffer: rows disjoint, the logits themselves or apart from them
inline int check_dlogits(const finetune_logits* in, const finetune_dlogits* out) {
  if (out == nullptr) return RDFFT_ERR_NULL;
  if (logit_rows(in) == 0) return RDFFT_OK;
  const int64_t ss = out->seq_stride, ps = out->pos_stride, v = in->vocab;
  if (!valid_strides(in, ss, ps)) return RDFFT_ERR_SHAPE;
  const bool one_seq = in->seqs == 1, one_pos = in->positions == 1;
  const bool by_seq = (one_pos || ps >= v) && (one_seq || ss >= (in->positions - 1) * ps + v);
  const bool by_pos = (one_seq || ss >= v) && (one_pos || ps >= (in->seqs - 1) * ss + v);
  if (!by_seq && !by_pos) return RDFFT_ERR_SHAPE;
  if (out->data == nullptr) return RDFFT_ERR_NULL;
  if (!aligned_to(out->data, dtype_bytes(int(in->dtype)))) return RDFFT_ERR_ALIGN;
  const Range o{out->data, logit_span(in, ss, ps) * dtype_bytes(int(in->dtype))};
  const bool same = out->data == in->data && (one_seq || ss == in->seq_stride) && (one_pos || ps == in->pos_stride);
  if ((!same && clashes(o, range_of(in))) || clashes(o, range_of_labels(in))) return RDFFT_ERR_ALIAS;
  return RDFFT_OK;
}

inline Range range_of(const finetune_logits* in, const finetune_dlogits* out) {
  if (out == nullptr) return {nullptr, 0};
  return {out->data, logit_span(in, out->seq_stride, out->pos_stride) * dtype_bytes(int(in->dtype))};
}

// fp32 arrays of a call: every one required to be there and aligned unless
// optional, outputs apart from each other and from all inputs
struct Array {
  const float* p;
  int64_t n;
  bool optional = false;
};
template <size_t NI, size_t NO>
inline int check_arrays(const finetune_logits* in, const finetune_dlogits* grad, const Array (&inputs)[NI],
                        const Array (&outputs)[NO], const void* ws, int64_t ws_need) {
  for (const Array& a : inputs)
    if (a.n > 0 && a.p == nullptr && !a.optional) return RDFFT_ERR_NULL;
  for (const Array& a : outputs)
    if (a.n > 0 && a.p == nullptr && !a.optional) return RDFFT_ERR_NULL;
  for (const Array& a : inputs)
    if (!aligned_to(a.p, 4)) return RDFFT_ERR_ALIGN;
  for (const Array& a : outputs)
    if (!aligned_to(a.p, 4)) return RDFFT_ERR_ALIGN;
  Range written[NO + 2];
  for (size_t i = 0; i < NO; ++i) written[i] = {outputs[i].p, outputs[i].n * 4};
  written[NO] = range_of(in, grad);
  written[NO + 1] = {ws, ws_need};
  for (size_t i = 0; i < NO + 2; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (clashes(written[i], written[j])) return RDFFT_ERR_ALIAS;
    for (const Array& a : inputs)
      if (clashes(written[i], Range{a.p, a.n * 4})) return RDFFT_ERR_ALIAS;
    if (i != NO && (clashes(written[i], range_of(in)) || clashes(written[i], range_of_labels(in))))
      return RDFFT_ERR_ALIAS;  // the gradient itself was checked by check_dlogits
  }
  return RDFFT_OK;
}

inline int check_preference(const finetune_logits* in, const finetune_preference* how) {
  if (how == nullptr) return RDFFT_ERR_NULL;
  if (in->seqs % 2 != 0) return RDFFT_ERR_SHAPE;
  if (how->kind < PREFERENCE_SIGMOID || how->kind > PREFERENCE_IPO || !(how->beta > 0.0) || isinf(how->beta) ||
      !(how->smoothing >= 0.0 && how->smoothing < 0.5))
    return RDFFT_ERR_SIZE;
  return RDFFT_OK;
}

inline int check_policy(const finetune_policy* how) {
  if (how == nullptr) return RDFFT_ERR_NULL;
  if (how->reduction < POLICY_TOKEN_MEAN || how->reduction > POLICY_SUM || !(how->clip_low >= 0.0) ||
      !(how->clip_high >= 0.0) || isnan(how->kl_coef) || isinf(how->kl_coef))
    return RDFFT_ERR_SIZE;
  return RDFFT_OK;
}

// ---- gradient tensors -----------------------------------------------------

inline int check_tensors(const finetune_tensor* t, int64_t n, bool with_out) {
  if (n < 0 || n > kMaxTensors) return RDFFT_ERR_SIZE;
  if (n > 0 && t == nullptr) return RDFFT_ERR_NULL;
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].dtype < 0 || t[i].dtype > 2) return RDFFT_ERR_DTYPE;
    if (t[i].count < 0 || t[i].count > kMaxElems || (total += t[i].count) > kMaxElems) return RDFFT_ERR_SIZE;
    if (t[i].count == 0) continue;
    const int64_t e = dtype_bytes(int(t[i].dtype));
    if (t[i].grad == nullptr || (with_out && t[i].out == nullptr)) return RDFFT_ERR_NULL;
    if (!aligned_to(t[i].grad, e) || (with_out && !aligned_to(t[i].out, e))) return RDFFT_ERR_ALIGN;
  }
  return RDFFT_OK;
}

// the norm and the workspace lie apart from each other and from every tensor
inline int check_norm_buffers(const finetune_tensor* t, int64_t n, bool with_out, const float* norm, const void* ws,
                              int64_t ws_bytes, int64_t need) {
  if (norm == nullptr) return RDFFT_ERR_NULL;
  if (!aligned_to(norm, 4)) return RDFFT_ERR_ALIGN;
  const int st = check_workspace(ws, ws_bytes, need);
  if (st != RDFFT_OK) return st;
  const Range rn{norm, 4}, rw{ws, need};
  if (clashes(rn, rw)) return RDFFT_ERR_ALIAS;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t bytes = t[i].count * dtype_bytes(int(t[i].dtype));
    const Range g{t[i].grad, bytes}, o{with_out ? t[i].out : nullptr, bytes};
    if (clashes(rn, g) || clashes(rn, o) || clashes(rw, g) || clashes(rw, o)) return RDFFT_ERR_ALIAS;
  }
  return RDFFT_OK;
}

// No element is written twice, and none is written that another tensor reads.
// Buffers that come in address order (a bucket's tensors, as they mostly do)
// are seen to be apart in one pass; any other order is sorted first.
inline int check_tensor_aliases(const finetune_tensor* t, int64_t n) {
  struct Piece {
    uintptr_t begin, end;
    bool written;
  };
  uintptr_t in_lo = UINTPTR_MAX, in_hi = 0, out_lo = UINTPTR_MAX, out_hi = 0;
  bool ordered = true, in_place = true, apart = true;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].count == 0) continue;
    const uintptr_t bytes = static_cast<uintptr_t>(t[i].count * dtype_bytes(int(t[i].dtype)));
    const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad), o = reinterpret_cast<uintptr_t>(t[i].out);
    if (o < out_hi) ordered = false;
    in_lo = std::min(in_lo, g), in_hi = std::max(in_hi, g + bytes);
    out_lo = std::min(out_lo, o), out_hi = std::max(out_hi, o + bytes);
    if (g != o) in_place = false;
  }
  apart = in_hi <= out_lo || out_hi <= in_lo;
  if (ordered && (in_place || apart)) return RDFFT_OK;
  Piece* p = new (std::nothrow) Piece[static_cast<size_t>(2 * n)];
  if (p == nullptr) return RDFFT_ERR_SIZE;
  int64_t m = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].count == 0) continue;
    const uintptr_t bytes = static_cast<uintptr_t>(t[i].count * dtype_bytes(int(t[i].dtype)));
    const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad), o = reinterpret_cast<uintptr_t>(t[i].out);
    if (g != o) p[m++] = {g, g + bytes, false};
    p[m++] = {o, o + bytes, true};
  }
  std::sort(p, p + m, [](const Piece& a, const Piece& b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;
  int st = RDFFT_OK;
  for (int64_t i = 0; i < m; ++i) {
    if (p[i].begin < (p[i].written ? any : written)) st = RDFFT_ERR_ALIAS;
    any = std::max(any, p[i].end);
    if (p[i].written) written = std::max(written, p[i].end);
  }
  delete[] p;
  return st;
}

}  // namespace finetune
