"""Inputs and error bounds shared by the tests of the sublayer operators.

Bounds are worst cases of the kernels' arithmetic, not fits.  With u = 2^-24
and a storage type of unit roundoff s (finetune_util.STORE):
  * a matrix product's sum of n terms errs by at most (n + 8) 2 u times the sum
    of magnitudes (2 u a term: the matrix unit may truncate);
  * a probability's exponent is formed from the score's sum, its scaling, the
    bias and the log-sum-exp, each rounded; its relative error is that of the
    exponent plus the function's own 2 ulp;
  * probabilities and ds are rounded to the storage type before a product
    (s each; half's are held 2^8 times as large, so what is lost below its
    smallest step is 2^-33), and results once more on store.
"""

from __future__ import annotations

import numpy as np
import torch

from oracle import attention_oracle as ao
from tests.finetune_util import STORE, U, f64, rng, store_err, stored

DEV = "cuda:0"
ROUND = {"f32": 0.0, "bf16": 2.0**-8, "f16": 2.0**-11}  # of an operand that is rounded for a product
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0**-33}


def inputs(key, b, tq, tk, hq, hk, d, dtype, spread=1.0):
    r = rng(77, *key)
    out = {}
    for name, shape in (("q", (b, tq, hq, d)), ("k", (b, tk, hk, d)), ("v", (b, tk, hk, d)), ("dout", (b, tq, hq, d))):
        t, ref = stored(spread * r.standard_normal(shape), dtype)
        out[name] = (t.to(DEV), ref)
    return out


def spans(key, b, tk):
    r = rng(78, *key)
    begin = r.integers(0, tk // 3 + 1, b)
    end = np.array([r.integers(lo, tk + 1) for lo in begin])
    if b > 1:
        end[-1] = begin[-1]  # a sequence without keys
    return begin.astype(np.int32), end.astype(np.int32)


def heads(t):
    return t.transpose(0, 2, 1, 3)


def score_error(q, k, scale, lse, bias=None):
    """Bound on the relative error of each probability, given the log-sum-exp that it is formed with."""
    g, d = q.shape[2] // k.shape[2], q.shape[3]
    kk = heads(np.repeat(k, g, axis=2))
    mag = np.matmul(np.abs(heads(q)), np.abs(kk).transpose(0, 1, 3, 2)) * scale
    top = np.where(np.isfinite(lse), np.abs(lse), 0.0)[..., None]
    extra = 0.0 if bias is None else np.abs(bias)
    return 2 * U * ((d + 8) * mag + 6 * (mag + extra + top) + 8)


def forward_bounds(q, k, v, scale, o, lse, p, dtype, bias=None):
    """(bound of o, bound of lse)."""
    g = q.shape[2] // k.shape[2]
    vv = np.abs(heads(np.repeat(v, g, axis=2)))
    e = score_error(q, k, scale, lse, bias)
    rel = np.where(p > 0, e, 0.0).max(-1, initial=0.0)  # of any term of a row
    n = k.shape[1]
    mass = np.matmul(p, vv)
    part = (ROUND[dtype] + 2 * rel[..., None] + (n + 16) * 2 * U) * mass + TINY[dtype] * vv.sum(2, keepdims=True)
    live = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return store_err(o, dtype) + heads(part), rel + (n + 16) * 2 * U + 4 * U * live + 2 * U


def backward_bounds(q, k, v, dout, scale, o, lse, p, ds, o_err, grads, dtype, bias=None):
    """Bounds of dq, dk, dv and of each ds that enters the bias's sums, where o was rounded to within o_err."""
    b, tq, hq, d = q.shape
    tk, hk = k.shape[1:3]
    g = hq // hk
    kk, vv = heads(np.repeat(k, g, axis=2)), heads(np.repeat(v, g, axis=2))
    qq, do = heads(q), heads(dout)
    e = np.where(p > 0, score_error(q, k, scale, lse, bias) + 2 * U * np.abs(np.where(np.isfinite(lse), lse, 0))[..., None], 0.0)
    mag = np.matmul(np.abs(do), np.abs(vv).transpose(0, 1, 3, 2))
    e_dp = (d + 8) * 2 * U * mag
    e_delta = (np.abs(do) * heads(o_err)).sum(-1) + (d + 8) * 2 * U * (np.abs(do) * np.abs(heads(o))).sum(-1)
    dp = np.matmul(do, vv.transpose(0, 1, 3, 2))
    delta = (p * dp).sum(-1)
    exact = ((tk + 8) * 2 * U + e.max(-1, initial=0.0)) * (p * mag).sum(-1) + (p * e_dp).sum(-1)
    base = np.abs(ds) * (e + 8 * U) + p * (e_dp + 4 * U * (mag + np.abs(delta)[..., None]))
    e_ds = base + p * np.maximum(e_delta, exact)[..., None]
    # half: ds is held times 2^-floor(log2) of the row's, or the largest row's, |dout|
    small = 0.0
    if dtype == "f16":
        small = 2.0**-24 * np.abs(do).max()
    r_ds = e_ds + ROUND[dtype] * (np.abs(ds) + e_ds) + np.where(p > 0, small, 0.0)
    gq, gk, gv = grads
    bq = scale * (np.matmul(r_ds, np.abs(kk)) + (tk + 8) * 2 * U * np.matmul(np.abs(ds), np.abs(kk)))
    n = g * tq

    def shared(t):
        return t.reshape(b, hk, g, tk, d).sum(2).transpose(0, 2, 1, 3)

    bk = shared(np.matmul(r_ds.transpose(0, 1, 3, 2), np.abs(qq))
                + (n + 8) * 2 * U * np.matmul(np.abs(ds).transpose(0, 1, 3, 2), np.abs(qq))) * scale
    r_p = p * (e + ROUND[dtype] + (n + 8) * 2 * U) + np.where(p > 0, TINY[dtype], 0.0)
    bv = shared(np.matmul(r_p.transpose(0, 1, 3, 2), np.abs(do)))
    return (store_err(gq, dtype) + heads(bq) + 4 * U * np.abs(gq), store_err(gk, dtype) + bk + 4 * U * np.abs(gk),
            store_err(gv, dtype) + bv + 4 * U * np.abs(gv), base + p * exact[..., None])


def case(key, b, tq, tk, hq, hk, d, dtype, causal=False, spanned=False, table=None, two_sided=True, distance=20,
         scale=None, spread=1.0):
    """Inputs, keyword arguments of the calls, and the oracle's view of them."""
    x = inputs(key, b, tq, tk, hq, hk, d, dtype, spread)
    how = dict(causal=causal, scale=d**-0.5 if scale is None else scale)
    begin = end = None
    if spanned:
        begin, end = spans(key, b, tk)
        how |= dict(key_begin=torch.from_numpy(begin).to(DEV), key_end=torch.from_numpy(end).to(DEV))
    bias = None
    if table:
        w, ref = stored(rng(79, *key).standard_normal((table, hq)), "f32")
        how |= dict(bias=w.to(DEV), max_distance=distance, bidirectional=two_sided)
        bias = ao.relative_bias(ref, tq, tk, distance, two_sided)
    return x, how, ao.visible(b, tq, tk, causal, begin, end), bias


__all__ = ["DEV", "STORE", "U", "ao", "backward_bounds", "case", "f64", "forward_bounds", "heads", "inputs", "rng",
           "score_error", "spans", "store_err", "stored"]
