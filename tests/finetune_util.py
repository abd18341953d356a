"""Inputs and error bounds shared by the tests of the fine-tuning operators.

Bounds are worst cases of the kernels' arithmetic, not fits.  With u = 2^-24
(fp32) and a storage type of unit roundoff s (2^-24, 2^-8 bfloat16, 2^-11
half; stores round once, so an output errs by s |value|, or by half the
smallest subnormal):
  * a sum of n terms by 64 or more threads errs by at most (n / 64 + 16) u
    times the sum of magnitudes;
  * exp(d) through exp2 errs by (|d| + 4) 2 u of its value (the product's
    rounding and the function's own 2 ulp).
"""

from __future__ import annotations

import numpy as np
import torch

U = 2.0**-24
STORE = {"f32": (2.0**-24, 2.0**-149), "bf16": (2.0**-8, 2.0**-134), "f16": (2.0**-11, 2.0**-25)}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
IGNORE = -100


def rng(*key):
    return np.random.default_rng(np.random.SeedSequence([4242, *[int(k) for k in key]]))


def stored(a, dtype):
    """(CPU tensor of `dtype`, float64 array of exactly its values)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to(TORCH[dtype])
    return t, t.to(torch.float64).numpy()


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def sum_err(n):
    return (n / 64 + 16) * U


def store_err(want, dtype):
    s, tiny = STORE[dtype]
    return s * np.abs(want) * 1.01 + tiny


def representable(want, dtype):
    """want with what rounds past the storage type's largest value as infinity (half: from 65520 on)."""
    return np.where(np.abs(want) >= 65520.0, np.copysign(np.inf, want), want) if dtype == "f16" else want


def within(got, want, bound):
    """Every element of got within bound of want (equal NaN and infinity included)."""
    got, want, bound = np.asarray(got, float), np.asarray(want, float), np.asarray(bound, float)
    same = (np.isnan(got) & np.isnan(want)) | (got == want)
    bad = ~(same | (np.abs(got - want) <= bound))
    if bad.any():
        i = tuple(int(k[0]) for k in np.nonzero(bad))
        b = np.broadcast_to(bound, want.shape)
        raise AssertionError(f"{int(bad.sum())} of {want.size} outside, first at {i}: got {got[i]!r} want {want[i]!r} "
                             f"bound {b[i]!r}")


def labels_of(r, n, t, v, masked=0.3, empty=()):
    lab = r.integers(0, v, size=(n, t))
    lab[r.random((n, t)) < masked] = IGNORE
    for s in empty:
        lab[s] = IGNORE
    return lab.astype(np.int64)


def logit_case(key, n, t, v, dtype, masked=0.3, empty=()):
    """(logits tensor, float64 logits, labels): rows of spread 3 with the label's logit raised."""
    r = rng(*key)
    lab = labels_of(r, n, t, v, masked, empty)
    x = 3.0 * r.standard_normal((n, t, v))
    for s, i in zip(*np.nonzero(lab != IGNORE)):
        x[s, i, lab[s, i]] += 6.0 * r.random()
    xt, xr = stored(x, dtype)
    return xt, xr, lab


def lse_err(logits, lse):
    """Bound on the error of a position's lse in fp32 storage."""
    v = logits.shape[-1]
    spread = np.max(np.abs(np.where(np.isfinite(logits), logits, 0.0)), axis=-1) * 2 + 4
    return sum_err(v) + (spread + 4) * 2 * U + 2 * U * np.abs(lse)


def grad_err(want, logits, labels, g, lse, dtype):
    """Bound on the error of g (onehot - softmax)."""
    d = np.abs(np.where(np.isfinite(logits), logits, 0.0) - lse[..., None])
    p = np.exp(np.minimum(logits - lse[..., None], 0.0))
    rel = lse_err(logits, lse)[..., None] + (d + 8) * 2 * U
    ag = np.abs(g)[..., None]
    return store_err(want, dtype) + ag * p * rel + 4 * U * np.abs(want) + ag * 2.0**-125
