"""float64 oracle of the fine-tuning operators (numpy, test infrastructure only).

Each function is the operator's formula written out; nothing here is shared
with the HIP path.
"""

from __future__ import annotations

import numpy as np

IGNORE = -100


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) of the rows of x."""
    mean = x.mean(axis=-1)
    mid = x - mean[..., None]
    rstd = 1.0 / np.sqrt((mid**2).mean(axis=-1) + eps)
    y = mid * rstd[..., None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_bwd(x, weight, mean, rstd, dy):
    """(dx, dw, db) from the given statistics; leading axes are all rows."""
    d = x.shape[-1]
    x, dy = x.reshape(-1, d), dy.reshape(-1, d)
    hat = (x - mean.reshape(-1, 1)) * rstd.reshape(-1, 1)
    g = dy if weight is None else dy * weight
    dx = rstd.reshape(-1, 1) * (g - g.mean(axis=1, keepdims=True) - hat * (g * hat).mean(axis=1, keepdims=True))
    return dx, (dy * hat).sum(axis=0), dy.sum(axis=0)


def token_logprob(logits, labels):
    """(logp, lse), 0 at ignored positions."""
    live = labels != IGNORE
    logp, lse = np.zeros(labels.shape), np.zeros(labels.shape)
    for s, i in zip(*np.nonzero(live)):
        row = logits[s, i].astype(np.float64)
        top = row.max()
        lse[s, i] = top + np.log(np.exp(row - top).sum())
        logp[s, i] = row[labels[s, i]] - lse[s, i]
    return logp, lse


def logits_grad(logits, labels, g):
    """g (per position) times (onehot - softmax); zero rows at ignored positions."""
    out = np.zeros(logits.shape)
    for s, i in zip(*np.nonzero(labels != IGNORE)):
        row = logits[s, i].astype(np.float64)
        p = np.exp(row - row.max())
        p /= p.sum()
        out[s, i] = -g[s, i] * p
        out[s, i, labels[s, i]] += g[s, i]
    return out


def _softplus(z):
    return np.logaddexp(0.0, z)


def preference(logp, labels, ref, beta, kind, smoothing=0.0, average=False):
    """(loss, logratio, d loss / d logp of each sequence's unmasked positions)."""
    live = labels != IGNORE
    n = labels.shape[0] // 2
    count = np.maximum(live.sum(axis=1), 1) if average else np.ones(2 * n)
    ratio = np.where(live, logp - ref, 0.0).sum(axis=1) / count
    h = ratio[:n] - ratio[n:]
    z = beta * h
    if kind == "sigmoid":
        loss = (1 - smoothing) * _softplus(-z) + smoothing * _softplus(z)
        dh = -beta * ((1 - smoothing) * np.exp(-_softplus(z)) - smoothing * np.exp(-_softplus(-z)))
    elif kind == "hinge":
        loss, dh = np.maximum(0.0, 1.0 - z), np.where(z < 1.0, -beta, 0.0)
    elif kind == "ipo":
        loss, dh = (h - 0.5 / beta) ** 2, 2.0 * (h - 0.5 / beta)
    else:
        raise ValueError(kind)
    return loss, ratio, np.concatenate([dh, -dh]) / count


def policy(logp, labels, old, adv, ref=None, low=0.2, high=0.2, kl_coef=0.0, reduction="token"):
    """(loss, kl, d loss / d logp); adv broadcasts over positions."""
    live = labels != IGNORE
    adv = np.broadcast_to(adv, labels.shape)
    r = np.exp(np.where(live, logp - old, 0.0))
    free, held = r * adv, np.clip(r, 1 - low, 1 + high) * adv
    each = -np.minimum(free, held)
    slope = np.where(free <= held, -free, 0.0)
    kl = np.zeros(labels.shape)
    if ref is not None:
        q = np.where(live, ref - logp, 0.0)
        kl = np.expm1(q) - q
        each, slope = each + kl_coef * kl, slope - kl_coef * np.expm1(q)
    if reduction == "token":
        w = live / max(1, live.sum())
    elif reduction == "sequence":
        w = live / np.maximum(1, live.sum(axis=1, keepdims=True)) / max(1, labels.shape[0])
    else:
        w = live.astype(np.float64)
    return (each * w).sum(), (kl * w).sum(), slope * w


def grad_norm(grads):
    return np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))


def clip(grads, max_norm, eps=1e-6):
    norm = grad_norm(grads)
    f = min(1.0, max_norm / (norm + eps))
    return norm, [g.astype(np.float64) * f for g in grads]
