/*
 * attention.h -- C ABI of the MI355X (gfx950) operators of a transformer
 * sublayer that store nothing of the size of the score matrix or of a mask
 * (libfinetune.so): attention whose backward recomputes the probabilities, a
 * learned relative position bias by buckets, and dropout from a counter-based
 * generator.
 *
 * The common rules are those of finetune.h: status codes and storage types,
 * caller-owned device pointers with the alignment of their element, workspaces
 * of the size a query gives (16-byte aligned), calls that only enqueue work,
 * arguments checked on the host before anything is enqueued, fixed orders of
 * summation.  Structs are host memory, read during the call.
 */
#ifndef ATTENTION_H
#define ATTENTION_H

#include <stdint.h>

#include "rdfft.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTENTION_ABI_VERSION 1

/* Version of this ABI (ATTENTION_ABI_VERSION of the library that was built). */
int attention_abi_version(void);

/* ---- relative position bias --------------------------------------------- */

/*
 * Buckets of relative positions r = key - query, the last query standing at
 * the last key.  Two-sided: the upper half of the buckets serves r > 0, the
 * lower half r <= 0, with n = |r|; one-sided: n = max(-r, 0).  With N buckets a
 * side, the first S = N / 2 (rounded down) are n itself; the others grow with
 * the logarithm,
 *     bucket = min(N - 1, S + floor(log(n / S) / log(max_distance / S) * (N - S))).
 * 2 <= N <= 256 a side (two-sided: count is even), S < max_distance <= 1024.
 */
typedef struct {
  int64_t count;        /* of buckets in all */
  int64_t max_distance; /* from here on all positions share the last bucket */
  int64_t two_sided;
} attention_buckets;

/*
 * relative_bias_fwd -- bias[h, i, j] = table[bucket(j - (i + keys - queries)), h].
 *   table [count, heads]           float
 *   bias  [heads, queries, keys]   dtype, written
 */
int relative_bias_fwd(const float* table, void* bias, int64_t heads, int64_t queries, int64_t keys,
                      const attention_buckets* buckets, int dtype, void* stream);

/* Bytes of the workspace of relative_bias_bwd. */
int relative_bias_workspace(int64_t batch, int64_t heads, int64_t queries, int64_t keys,
                            const attention_buckets* buckets, int64_t* bytes);

/*
 * relative_bias_bwd -- dtable[c, h] = sum of dbias[b, h, i, j] over the batch
 * and the positions of bucket c.
 *   dbias  [batch, heads, queries, keys]  dtype; strides count elements, keys contiguous
 *   dtable [count, heads]                 float, overwritten
 */
int relative_bias_bwd(const void* dbias, int64_t batch_stride, int64_t head_stride, int64_t query_stride,
                      float* dtable, int64_t batch, int64_t heads, int64_t queries, int64_t keys,
                      const attention_buckets* buckets, void* ws, int64_t ws_bytes, int dtype, void* stream);

/* ---- attention ---------------------------------------------------------- */

/* Shapes and rules of an attention call. */
typedef struct {
  int64_t batch, queries, keys;
  int64_t heads, kv_heads; /* heads is a multiple of kv_heads: query head h reads key head h / (heads / kv_heads) */
  int64_t head_dim;        /* 1 .. 128 */
  int64_t dtype;
  double scale;            /* > 0 */
  int64_t causal;          /* nonzero: query i sees keys j <= i + keys - queries */
  const int32_t* key_begin; /* [batch] or NULL (0): the keys [begin, end) of a sequence count, */
  const int32_t* key_end;   /* [batch] or NULL (keys); the others are not read.  Values are clamped to 0 .. keys */
  const float* bias;        /* [buckets.count, heads] or NULL: added to the scaled scores by bucket */
  attention_buckets buckets; /* read when bias is given */
} attention_problem;

/* Tokens by heads: element (b, t, h, x) at data[b * batch_stride + t * token_stride + h * head_stride + x]. */
typedef struct {
  void* data;
  int64_t batch_stride, token_stride, head_stride; /* elements, >= 0 */
} attention_tensor;

/* Bytes of the workspace of attention_fwd (backward = 0) or attention_bwd (1). */
int attention_workspace(const attention_problem* a, int backward, int64_t* bytes);

/*
 * attention_fwd -- with s_ij = scale q_i . k_j + bias and the softmax over the
 * keys j that query i sees,
 *     lse_i = log sum_j exp s_ij,  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j.
 * A query that sees no key gets o = 0 and lse = -infinity.
 *   q [batch, queries, heads, head_dim], k, v [batch, keys, kv_heads, head_dim]
 *   o   like q, written; must not overlap q, k, v
 *   lse [batch, heads, queries]  float, written
 * Products take the storage type with fp32 sums; p is rounded to the storage
 * type for its product with v.  Infinities and NaN of keys and values that some
 * query sees may also reach queries nearby that do not see them (0 times them).
 */
int attention_fwd(const attention_problem* a, const attention_tensor* q, const attention_tensor* k,
                  const attention_tensor* v, const attention_tensor* o, float* lse, void* ws, int64_t ws_bytes,
                  void* stream);

/*
 * attention_bwd -- gradients for an upstream gradient dout of o, from the
 * forward's o and lse; the probabilities are computed again:
 *     dp_ij = dout_i . v_j,  delta_i = sum_j p_ij dp_ij,  ds_ij = p_ij (dp_ij - delta_i),
 *     dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i,
 *     dbias[c, h] = sum of ds over the batch and the positions of bucket c.
 * dk and dv sum over the query heads that share a key head.  Keys outside a
 * sequence's span get zeros; dout of queries that see no key is not used.
 *   dq like q, dk and dv like k: written, none overlapping another tensor
 *   dbias [buckets.count, heads]  float, overwritten, or NULL
 */
int attention_bwd(const attention_problem* a, const attention_tensor* q, const attention_tensor* k,
                  const attention_tensor* v, const attention_tensor* o, const float* lse,
                  const attention_tensor* dout, const attention_tensor* dq, const attention_tensor* dk,
                  const attention_tensor* dv, float* dbias, void* ws, int64_t ws_bytes, void* stream);

/* ---- dropout ------------------------------------------------------------ */

/*
 * The mask of element e (its index in row-major order, rows * d in all) is 16
 * bits of the counter-based generator Philox4x32-10 (Salmon, Moraes, Dror and
 * Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): counter words
 * (low, high word of e / 8; low, high word of offset), key words (low, high
 * word of seed); output word (e % 8) / 2, its low half for even e.  The element
 * is dropped where these bits are below round(65536 p), and kept ones are
 * scaled by 65536 / (65536 - round(65536 p)), so that the mean is kept exactly.
 */
typedef struct {
  double p;                /* 0 .. 1 */
  uint64_t seed, offset;
  const uint64_t* device_seed; /* device memory or NULL: added to seed when the kernel runs (replays of a graph) */
} attention_dropout;

/*
 * dropout_fwd -- y = residual + (kept ? x * scale : 0).
 *   x, residual, y [rows, d]  dtype, rows their stride apart (>= d); residual may be NULL;
 *                  y may be x or residual (same pointer and stride), else must not overlap them
 */
int dropout_fwd(const void* x, const void* residual, void* y, int64_t rows, int64_t d, int64_t x_stride,
                int64_t residual_stride, int64_t y_stride, const attention_dropout* how, int dtype, void* stream);

/* dropout_bwd -- dx = kept ? dy * scale : 0 with the forward's mask; dx may be dy itself. */
int dropout_bwd(const void* dy, void* dx, int64_t rows, int64_t d, int64_t dy_stride, int64_t dx_stride,
                const attention_dropout* how, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTENTION_H */
