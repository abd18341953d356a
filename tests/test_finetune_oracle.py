"""Pins of the fine-tuning oracle: its gradients against central differences,
and its values against torch's float64 functions (CPU only)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import finetune_oracle as fo
from tests.finetune_util import IGNORE, labels_of, rng


def _differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f(x)
        x[i] = keep - h
        g[i] = (up - f(x)) / (2 * h)
        x[i] = keep
    return g


# central differences of step 1e-5 in float64: truncation h^2 f''' / 6 ~ 1e-10 f''' and rounding 1e-16 f / h ~ 1e-11 f
DIFF = 1e-7


def test_layer_norm_values_and_differences():
    r = rng(1)
    x, w, b, dy = r.standard_normal((3, 7)) + 2.0, r.standard_normal(7), r.standard_normal(7), r.standard_normal((3, 7))
    y, mean, rstd = fo.layer_norm(x, w, b, 1e-3)
    want = torch.nn.functional.layer_norm(torch.from_numpy(x), (7,), torch.from_numpy(w), torch.from_numpy(b), 1e-3)
    assert np.allclose(y, want.numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, db = fo.layer_norm_bwd(x, w, mean, rstd, dy)
    assert np.allclose(dx, _differences(lambda v: (fo.layer_norm(v, w, b, 1e-3)[0] * dy).sum(), x), atol=DIFF)
    assert np.allclose(dw, _differences(lambda v: (fo.layer_norm(x, v, b, 1e-3)[0] * dy).sum(), w), atol=DIFF)
    assert np.allclose(db, _differences(lambda v: (fo.layer_norm(x, w, v, 1e-3)[0] * dy).sum(), b), atol=DIFF)


def _logits(n=4, t=3, v=5):
    r = rng(2)
    return r, 2.0 * r.standard_normal((n, t, v)), labels_of(r, n, t, v, 0.3, empty=(2,))


def test_token_logprob():
    _, x, lab = _logits()
    logp, lse = fo.token_logprob(x, lab)
    want = torch.log_softmax(torch.from_numpy(x), -1).gather(2, torch.from_numpy(lab).clamp(min=0)[..., None])[..., 0]
    live = lab != IGNORE
    assert np.allclose(logp[live], want.numpy()[live], rtol=1e-13) and not logp[~live].any()
    assert np.allclose(lse[live], torch.logsumexp(torch.from_numpy(x), -1).numpy()[live], rtol=1e-13)


@pytest.mark.parametrize("kind,smoothing", [("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_differences(kind, smoothing, average):
    r, x, lab = _logits()
    ref = fo.token_logprob(x, lab)[0] + 0.5 * r.standard_normal(lab.shape)

    def total(v):
        return fo.preference(fo.token_logprob(v, lab)[0], lab, ref, 0.3, kind, smoothing, average)[0].sum()

    slope = fo.preference(fo.token_logprob(x, lab)[0], lab, ref, 0.3, kind, smoothing, average)[2]
    got = fo.logits_grad(x, lab, np.broadcast_to(slope[:, None], lab.shape))
    assert np.allclose(got, _differences(total, x), atol=DIFF)


@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("with_ref", [False, True])
def test_policy_differences(reduction, with_ref):
    r, x, lab = _logits()
    logp = fo.token_logprob(x, lab)[0]
    old, adv = logp + 0.3 * r.standard_normal(lab.shape), r.standard_normal((4, 1))
    ref = logp + 0.3 * r.standard_normal(lab.shape) if with_ref else None
    kw = dict(ref=ref, low=0.1, high=0.25, kl_coef=0.2, reduction=reduction)

    def total(v):
        return fo.policy(fo.token_logprob(v, lab)[0], lab, old, adv, **kw)[0]

    slope = fo.policy(logp, lab, old, adv, **kw)[2]
    assert np.allclose(fo.logits_grad(x, lab, slope), _differences(total, x), atol=DIFF)


def test_clip():
    r = rng(3)
    grads = [r.standard_normal(5), r.standard_normal((2, 3)), np.zeros(0)]
    norm, out = fo.clip(grads, 0.5)
    assert np.isclose(norm, torch.cat([torch.from_numpy(g).flatten() for g in grads]).norm().item(), rtol=1e-14)
    assert np.isclose(fo.grad_norm(out), 0.5, rtol=1e-5)
    assert all(np.array_equal(a, b) for a, b in zip(fo.clip(grads, 1e3)[1], grads))
