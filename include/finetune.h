/*
 * finetune.h -- C ABI of the MI355X (gfx950) operators around the circulant
 * layers in a fine-tuning step (libfinetune.so): layer normalisation, token
 * log-probabilities, the pairwise preference loss and the clipped policy loss
 * on vocabulary logits, and the global gradient norm with clipping.
 *
 * Common rules for every entry point
 *   - Status codes and storage types are those of rdfft.h (RDFFT_OK,
 *     RDFFT_ERR_*, RDFFT_F32 / RDFFT_BF16 / RDFFT_F16); RDFFT_ERR_SIZE: a
 *     count or a parameter outside its range, or a workspace too small;
 *     RDFFT_ERR_SHAPE: strides or counts that do not go together.
 *   - Pointers are DEVICE pointers owned by the caller unless marked "host".
 *     They need the alignment of their element only.  Rows of activations and
 *     logits may be strided (strides count elements); everything else is
 *     contiguous.  The library allocates no device memory and keeps no
 *     per-call state; where a call needs a workspace the caller passes one of
 *     the size its query gives (16-byte aligned; contents do not matter).
 *   - `stream` is a hipStream_t (NULL = the null stream).  Calls only enqueue
 *     work and return, and can be captured into a graph.
 *   - Arguments are checked on the host before anything is enqueued.  On any
 *     error the call returns a nonzero status and neither reads nor writes
 *     device memory.
 *   - Arithmetic is fp32 with fp64 for long sums of few values; 16-bit results
 *     are rounded to nearest even once, on store.  Every sum has a fixed
 *     order: results are bitwise the same from call to call.
 *   - Non-finite inputs are propagated, not checked.
 */
#ifndef FINETUNE_H
#define FINETUNE_H

#include <stdint.h>

#include "rdfft.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FINETUNE_ABI_VERSION 1

/* Version of this ABI (FINETUNE_ABI_VERSION of the library that was built). */
int finetune_abi_version(void);

/* Static string naming a status code of the calls below. */
const char* finetune_status_string(int status);

/* ---- layer normalisation ------------------------------------------------ */

/*
 * layer_norm_fwd -- for every row x of d elements
 *     mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
 *     y = (x - mean) * rstd * weight + bias.
 *   x       [rows, d]  dtype, rows x_stride elements apart (>= d)
 *   weight  [d]        float or NULL (1)
 *   bias    [d]        float or NULL (0)
 *   y       [rows, d]  dtype, rows y_stride apart, written; may be x itself
 *                      (same pointer and stride), else must not overlap it
 *   mean, rstd [rows]  float, written; may be NULL
 * 1 <= d <= 2^20; eps >= 0.  rows == 0 is a no-op.
 */
int layer_norm_fwd(const void* x, const float* weight, const float* bias, void* y, float* mean, float* rstd,
                   int64_t rows, int64_t d, int64_t x_stride, int64_t y_stride, double eps, int dtype, void* stream);

/* Bytes of the workspace layer_norm_bwd needs (0 without the weight sums). */
int layer_norm_bwd_workspace(int64_t rows, int64_t d, int64_t* bytes);

/*
 * layer_norm_bwd -- gradients of layer_norm_fwd for an upstream gradient dy,
 * from the saved mean and rstd.  With hat = (x - mean) rstd and g = dy weight:
 *     dx = rstd (g - mean_d(g) - hat mean_d(g hat)),
 *     dweight = sum over rows of dy hat,  dbias = sum over rows of dy.
 *   dx       [rows, d]  dtype, rows dx_stride apart, written; may be NULL, or
 *                       dy itself (same pointer and stride)
 *   dweight  [d]        float, overwritten; may be NULL
 *   dbias    [d]        float, overwritten; may be NULL
 *   ws       workspace of ws_bytes, needed when dweight or dbias is given
 * At least one of dx, dweight, dbias is required.  When rows == 0, dweight and
 * dbias are set to zero.
 */
int layer_norm_bwd(const void* x, const float* weight, const float* mean, const float* rstd, const void* dy, void* dx,
                   float* dweight, float* dbias, void* ws, int64_t ws_bytes, int64_t rows, int64_t d,
                   int64_t x_stride, int64_t dy_stride, int64_t dx_stride, int dtype, void* stream);

/* ---- losses on vocabulary logits ---------------------------------------- */

/* label of a position that takes no part: its logits are not read */
#define FINETUNE_IGNORE (-100)

/*
 * Logits and labels of a batch of sequences (host struct, read during the
 * call).  The logits of position i of sequence s are the `vocab` contiguous
 * elements from data + s * seq_stride + i * pos_stride; labels[s, i] is the
 * token whose log-probability they give.  A label that is neither
 * FINETUNE_IGNORE nor in [0, vocab) makes its position's values NaN (nothing
 * out of range is read).  1 <= vocab <= 2^24, seqs * positions < 2^31.
 */
typedef struct {
  const void* data;
  const int64_t* labels; /* [seqs, positions] */
  int64_t seqs, positions, vocab;
  int64_t seq_stride, pos_stride; /* >= 0 */
  int64_t dtype;
} finetune_logits;

/*
 * A gradient of the logits: [seqs, positions, vocab] of the logits' dtype with
 * strides of its own, rows disjoint.  `data` may be the logits themselves
 * (same pointer and strides: the gradient replaces them), else must not
 * overlap them.  Ignored positions get zeros.
 */
typedef struct {
  void* data;
  int64_t seq_stride, pos_stride;
} finetune_dlogits;

/* Bytes of the workspace of the calls below for this shape (pointers unread). */
int finetune_logits_workspace(const finetune_logits* in, int64_t* bytes);

/*
 * token_logprob -- logp = x[label] - lse, lse = log sum_j exp x_j.
 *   logp [seqs, positions]  float, written; 0 at ignored positions
 *   lse  [seqs, positions]  float, written; 0 at ignored positions
 */
int token_logprob(const finetune_logits* in, float* logp, float* lse, void* ws, int64_t ws_bytes, void* stream);

/*
 * token_logprob_bwd -- dlogits = dlogp (onehot(label) - exp(x - lse)).
 *   lse, dlogp [seqs, positions]  float
 */
int token_logprob_bwd(const finetune_logits* in, const float* lse, const float* dlogp, const finetune_dlogits* out,
                      void* stream);

#define PREFERENCE_SIGMOID 0 /* -(1-e) log sigma(b h) - e log sigma(-b h); e = 0: the first term alone */
#define PREFERENCE_HINGE 1   /* max(0, 1 - b h) */
#define PREFERENCE_IPO 2     /* (h - 1/(2 b))^2 */

typedef struct {
  int64_t kind;     /* PREFERENCE_* */
  int64_t average;  /* nonzero: log-ratios are means over a sequence's unmasked positions, else sums */
  double beta;      /* b > 0 */
  double smoothing; /* e in [0, 1/2); only PREFERENCE_SIGMOID has a use for it */
} finetune_preference;

/*
 * preference_loss_fwd -- paired log-ratio loss.  Sequences 0..n-1 are the
 * chosen answers and n..2n-1 the rejected ones (in->seqs = 2n).  With
 * logratio_s = sum (or mean) over the unmasked positions of logp - ref_logp
 * and h = logratio_chosen - logratio_rejected, loss is the kind's function.
 *   ref_logp [2n, positions]  float, the reference model's token log-probs
 *   loss     [n]              float, written
 *   logratio [2n]             float, written (0 for a sequence masked entirely)
 *   logp, lse [2n, positions] float, written as by token_logprob
 *   slope    [2n]             float, written: d loss / d logp of every
 *                             unmasked position of the sequence
 */
int preference_loss_fwd(const finetune_logits* in, const float* ref_logp, const finetune_preference* how, float* loss,
                        float* logratio, float* logp, float* lse, float* slope, void* ws, int64_t ws_bytes,
                        void* stream);

/*
 * preference_loss_bwd -- the logits' gradient of sum_b dloss[b] loss[b] from
 * the forward's lse and slope.
 *   dloss [n] float
 */
int preference_loss_bwd(const finetune_logits* in, const float* lse, const float* slope, const float* dloss,
                        const finetune_dlogits* out, void* stream);

/*
 * preference_loss_step -- forward and the logits' gradient of
 * scale * sum_b loss[b] in one call.
 */
int preference_loss_step(const finetune_logits* in, const float* ref_logp, const finetune_preference* how,
                         double scale, float* loss, float* logratio, float* logp, float* lse, float* slope,
                         const finetune_dlogits* out, void* ws, int64_t ws_bytes, void* stream);

#define POLICY_TOKEN_MEAN 0    /* mean over all unmasked positions */
#define POLICY_SEQUENCE_MEAN 1 /* mean over the sequences of the mean over their unmasked positions */
#define POLICY_SUM 2           /* sum over all unmasked positions */

typedef struct {
  int64_t reduction;           /* POLICY_* */
  int64_t advantage_per_token; /* advantages are [seqs, positions], else [seqs] */
  double clip_low, clip_high;  /* ratio clipped to [1 - clip_low, 1 + clip_high]; both >= 0 */
  double kl_coef;              /* k */
} finetune_policy;

/*
 * policy_loss_fwd -- clipped policy loss with a KL term.  Per unmasked position
 *     r = exp(logp - old_logp),  q = ref_logp - logp,  kl = exp(q) - q - 1,
 *     l = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + k kl,
 * reduced over positions (a sequence without any counts as 0).
 *   old_logp [seqs, positions]  float
 *   ref_logp [seqs, positions]  float or NULL (kl = 0)
 *   advantages                  float, see finetune_policy
 *   stats    [2]                float, written: the loss, and kl reduced likewise
 *   logp, lse [seqs, positions] float, written as by token_logprob
 *   slope    [seqs, positions]  float, written: d loss / d logp
 */
int policy_loss_fwd(const finetune_logits* in, const float* old_logp, const float* ref_logp, const float* advantages,
                    const finetune_policy* how, float* stats, float* logp, float* lse, float* slope, void* ws,
                    int64_t ws_bytes, void* stream);

/*
 * policy_loss_bwd -- the logits' gradient of dloss[0] * loss from the
 * forward's lse and slope.
 *   dloss [1] float
 */
int policy_loss_bwd(const finetune_logits* in, const float* lse, const float* slope, const float* dloss,
                    const finetune_dlogits* out, void* stream);

/* policy_loss_step -- forward and the logits' gradient of scale * loss in one call. */
int policy_loss_step(const finetune_logits* in, const float* old_logp, const float* ref_logp, const float* advantages,
                     const finetune_policy* how, double scale, float* stats, float* logp, float* lse, float* slope,
                     const finetune_dlogits* out, void* ws, int64_t ws_bytes, void* stream);

/* ---- global gradient norm and clipping ---------------------------------- */

/* One gradient tensor (an element of a host array, read during the call). */
typedef struct {
  const void* grad; /* count elements of dtype */
  void* out;        /* clipped values, same type; grad itself, or not overlapping any grad or other out */
  int64_t count;    /* >= 0 */
  int64_t dtype;
} finetune_tensor;

/* Bytes of the workspace of grad_norm and clip_grad_norm for these tensors (`out` unread). */
int grad_norm_workspace(const finetune_tensor* tensors, int64_t n, int64_t* bytes);

/* grad_norm -- norm[0] = sqrt(sum of g^2 over all tensors) (`out` unread). */
int grad_norm(const finetune_tensor* tensors, int64_t n, float* norm, void* ws, int64_t ws_bytes, void* stream);

/*
 * clip_grad_norm -- norm as above, and out = g * min(1, max_norm / (norm + eps))
 * for every tensor.  A norm that is not finite makes the factor 0 or NaN, as
 * the formula has it.  max_norm >= 0, eps >= 0.
 */
int clip_grad_norm(const finetune_tensor* tensors, int64_t n, double max_norm, double eps, float* norm, void* ws,
                   int64_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FINETUNE_H */
