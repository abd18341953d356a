// attention_validate.hpp -- host-side argument checks of attention.h (no HIP calls).
//
// Every entry point runs these before enqueuing anything; on failure it
// returns the status and touches no device memory.
#pragma once

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "attention.h"
#include "validate.hpp"

namespace finetune {

constexpr int64_t kMaxTokens = int64_t(1) << 24;  // queries or keys of a sequence
constexpr int64_t kMaxHeadDim = 128;
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;  // of a launch: HIP takes fewer than 2^32 threads

inline int check_buckets(const attention_buckets* b) {
  if (b == nullptr) return RDFFT_ERR_NULL;
  if (b->count < 2 || b->count > 512 || (b->two_sided && b->count % 2)) return RDFFT_ERR_SIZE;
  const int64_t side = b->two_sided ? b->count / 2 : b->count;
  if (side < 2 || side > 256 || b->max_distance <= side / 2 || b->max_distance > 1024) return RDFFT_ERR_SIZE;
  return RDFFT_OK;
}

inline bool valid_dims(int64_t batch, int64_t heads, int64_t tq, int64_t tk) {
  return batch >= 0 && heads >= 1 && tq >= 0 && tk >= 0 && tq <= kMaxTokens && tk <= kMaxTokens &&
         heads <= kMaxTokens && batch <= kMaxTokens && batch * heads <= kMaxTokens;
}

// ---- relative position bias -----------------------------------------------

inline int check_bias_fwd(const float* table, const void* bias, int64_t heads, int64_t tq, int64_t tk,
                          const attention_buckets* b, int dtype) {
  if (!valid_dtype(dtype)) return RDFFT_ERR_DTYPE;
  const int st = check_buckets(b);
  if (st != RDFFT_OK) return st;
  if (!valid_dims(1, heads, tq, tk) || tq * tk > kMaxElems / heads) return RDFFT_ERR_SIZE;
  if (tq == 0 || tk == 0) return RDFFT_OK;
  if (table == nullptr || bias == nullptr) return RDFFT_ERR_NULL;
  const int64_t e = dtype_bytes(dtype);
  if (!aligned_to(table, 4) || !aligned_to(bias, e)) return RDFFT_ERR_ALIGN;
  if (overlaps(table, b->count * heads * 4, bias, heads * tq * tk * e)) return RDFFT_ERR_ALIAS;
  return RDFFT_OK;
}

// whether sizes and strides (>= 0) keep every offset below the element limit
inline bool valid_strides(const int64_t (&size)[3], const int64_t (&stride)[3]) {
  int64_t span = 0;
  for (int n = 0; n < 3; ++n) {
    if (stride[n] < 0) return false;
    if (size[n] <= 1) continue;
    if (stride[n] > kMaxElems / size[n]) return false;
    span += stride[n] * (size[n] - 1);
  }
  return span <= kMaxElems;
}
inline int64_t elements(const int64_t (&size)[3], const int64_t (&stride)[3], int64_t row) {
  int64_t n = row;
  for (int k = 0; k < 3; ++k) {
    if (size[k] == 0) return 0;
    n += stride[k] * (size[k] - 1);
  }
  return n;
}

inline int check_bias_bwd(const void* dbias, const int64_t (&stride)[3], const float* dtable, int64_t batch,
                          int64_t heads, int64_t tq, int64_t tk, const attention_buckets* b, const void* ws,
                          int64_t ws_bytes, int64_t need, int dtype) {
  if (!valid_dtype(dtype)) return RDFFT_ERR_DTYPE;
  int st = check_buckets(b);
  if (st != RDFFT_OK) return st;
  if (!valid_dims(batch, heads, tq, tk)) return RDFFT_ERR_SIZE;
  if (dtable == nullptr) return RDFFT_ERR_NULL;
  if (!aligned_to(dtable, 4)) return RDFFT_ERR_ALIGN;
  st = check_workspace(ws, ws_bytes, need);
  if (st != RDFFT_OK) return st;
  const int64_t out = b->count * heads * 4;
  if (overlaps(dtable, out, ws, need)) return RDFFT_ERR_ALIAS;
  if (batch == 0 || tq == 0 || tk == 0) return RDFFT_OK;
  const int64_t size[3] = {batch, heads, tq};
  if (!valid_strides(size, stride)) return RDFFT_ERR_SHAPE;
  if (dbias == nullptr) return RDFFT_ERR_NULL;
  const int64_t e = dtype_bytes(dtype), bytes = elements(size, stride, tk) * e;
  if (!aligned_to(dbias, e)) return RDFFT_ERR_ALIGN;
  if (overlaps(dbias, bytes, dtable, out) || overlaps(dbias, bytes, ws, need)) return RDFFT_ERR_ALIAS;
  return RDFFT_OK;
}

// ---- attention ------------------------------------------------------------

inline int check_problem(const attention_problem* a) {
  if (a == nullptr) return RDFFT_ERR_NULL;
  if (a->dtype < 0 || a->dtype > 2 || !valid_dtype(static_cast<int>(a->dtype))) return RDFFT_ERR_DTYPE;
  if (!valid_dims(a->batch, a->heads, a->queries, a->keys) || a->kv_heads < 1 || a->head_dim < 1 ||
      a->head_dim > kMaxHeadDim)
    return RDFFT_ERR_SIZE;
  if (a->kv_heads > a->heads || a->heads % a->kv_heads) return RDFFT_ERR_SHAPE;
  const float scale = static_cast<float>(a->scale);
  if (!(a->scale > 0.0) || !(scale > 0.0f) || !isfinite(scale * 1.5f)) return RDFFT_ERR_SIZE;
  if (!aligned_to(a->key_begin, 4) || !aligned_to(a->key_end, 4) || !aligned_to(a->bias, 4)) return RDFFT_ERR_ALIGN;
  return a->bias ? check_buckets(&a->buckets) : RDFFT_OK;
}

// A tensor of `tokens` x `heads` rows for each sequence: its shape with its strides
struct Rows4 {
  const void* p;
  int64_t size[3], stride[3];  // batch, tokens, heads
  int64_t d, bytes_each, bytes;
  bool empty() const { return size[0] == 0 || size[1] == 0; }
};
inline Rows4 rows4(const attention_problem& a, const attention_tensor& t, bool keys) {
  Rows4 r{t.data,
          {a.batch, keys ? a.keys : a.queries, keys ? a.kv_heads : a.heads},
          {t.batch_stride, t.token_stride, t.head_stride},
          a.head_dim,
          dtype_bytes(static_cast<int>(a.dtype)),
          0};
  return r;
}

inline int check_tensor(Rows4& r, bool written) {
  if (r.empty()) return RDFFT_OK;
  if (!valid_strides(r.size, r.stride)) return RDFFT_ERR_SHAPE;
  if (written) {  // no two elements at one place: each stride reaches past what lies inside it
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return r.stride[x] < r.stride[y]; });
    int64_t extent = r.d;
    for (int n : order) {
      if (r.size[n] <= 1) continue;
      if (r.stride[n] < extent) return RDFFT_ERR_SHAPE;
      extent += r.stride[n] * (r.size[n] - 1);
    }
  }
  if (r.p == nullptr) return RDFFT_ERR_NULL;
  if (!aligned_to(r.p, r.bytes_each)) return RDFFT_ERR_ALIGN;
  r.bytes = elements(r.size, r.stride, r.d) * r.bytes_each;
  return RDFFT_OK;
}

// Whether two tensors may share memory.  Parts of one buffer that interleave token by token (the heads of q, k and v
// in a fused projection) do not: equal token strides, sequences a whole number of tokens apart, and rows that stay
// beside each other in a token's stretch.
inline bool clash(const Rows4& x, const Rows4& y) {
  if (x.empty() || y.empty() || !overlaps(x.p, x.bytes, y.p, y.bytes)) return false;
  const int64_t st = x.stride[1];
  if (st <= 0 || y.stride[1] != st) return true;
  for (const Rows4* r : {&x, &y})
    if ((r->size[0] > 1 && r->stride[0] % st) || (r->size[2] - 1) * r->stride[2] + r->d > st) return true;
  const int64_t e = x.bytes_each, step = st * e;
  int64_t gap = (reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p)) % step;
  if (gap < 0) gap += step;
  const int64_t wx = ((x.size[2] - 1) * x.stride[2] + x.d) * e, wy = ((y.size[2] - 1) * y.stride[2] + y.d) * e;
  return gap < wx || gap + wy > step;
}
inline bool clash(const Rows4& x, const void* p, int64_t bytes) {
  return !x.empty() && overlaps(x.p, x.bytes, p, bytes);
}

// ---- dropout --------------------------------------------------------------

inline int check_dropout(const void* x, const void* res, const void* y, int64_t rows, int64_t d, int64_t xs,
                         int64_t rs, int64_t ys, const attention_dropout* how, int dtype) {
  if (!valid_dtype(dtype)) return RDFFT_ERR_DTYPE;
  if (how == nullptr) return RDFFT_ERR_NULL;
  if (!(how->p >= 0.0 && how->p <= 1.0) || d < 1 || rows < 0 || rows > kMaxElems / d) return RDFFT_ERR_SIZE;
  if (rows == 0) return RDFFT_OK;
  if (!valid_rows(rows, d, xs) || !valid_rows(rows, d, ys) || (res && !valid_rows(rows, d, rs)))
    return RDFFT_ERR_SHAPE;
  if (x == nullptr || y == nullptr) return RDFFT_ERR_NULL;
  const int64_t e = dtype_bytes(dtype);
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(res, e) || !aligned_to(how->device_seed, 8))
    return RDFFT_ERR_ALIGN;
  const int64_t out = span(rows, d, ys) * e;
  if (!(x == y && xs == ys) && overlaps(y, out, x, span(rows, d, xs) * e)) return RDFFT_ERR_ALIAS;
  if (res && !(res == y && rs == ys) && overlaps(y, out, res, span(rows, d, rs) * e)) return RDFFT_ERR_ALIAS;
  if (overlaps(y, out, how->device_seed, 8)) return RDFFT_ERR_ALIAS;
  return RDFFT_OK;
}

}  // namespace finetune
