"""GPU tests of the fine-tuning operators at the edges of fp32: rows of logits
with a common offset or at a type's lowest value, log-ratios that are infinite,
and normalised rows whose mean is large.

With u = 2^-24: exp(x - lse) takes one rounding of x - lse, one of its product
with log2(e) and the constant's own (0.22 u), so the exponent errs by less than
2.5 u |x - lse| and the value by that and a few roundings of its own; 3 u |x -
lse| + 8 u is asked for.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import block_circulant_layers_amd as bcl
from tests.finetune_util import IGNORE, STORE, TORCH, U, f64, rng, stored, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LOWEST = {dt: float(torch.finfo(TORCH[dt]).min) for dt in TORCH}


def check_gradient(got, x, lab, lse, g, dtype):
    """got against g (onehot - exp(x - lse)) in float64 at the same float32 lse."""
    x, lse, g = f64(x), f64(lse)[..., None], np.asarray(g, np.float64)[..., None]
    d = x - lse
    p = np.where(lab[..., None] == IGNORE, 0.0, np.exp(np.where(lab[..., None] == IGNORE, 0.0, d)))
    hot = np.arange(x.shape[-1]) == lab[..., None]
    want = np.where(lab[..., None] == IGNORE, 0.0, g * (hot - p))
    s, tiny = STORE[dtype]
    within(f64(got), want, s * np.abs(want) * 1.01 + tiny + np.abs(g) * p * (3 * np.abs(d) + 8) * U + 4 * U * np.abs(want)
           + np.abs(g) * 2.0**-125)


def offset_case(n, t, v, offset, dtype):
    """Logits around `offset` ("lowest": nothing but the type's lowest value) and labels, some masked."""
    r = rng(200, n, t, v)
    lab = r.integers(0, v, size=(n, t))
    lab[r.random((n, t)) < 0.2] = IGNORE
    lab[:, 0] = v // 2  # an unmasked position in every sequence
    x = np.full((n, t, v), LOWEST[dtype]) if offset == "lowest" else offset + 3.0 * r.standard_normal((n, t, v))
    return stored(x, dtype)[0].to(DEV), torch.from_numpy(lab).to(DEV), lab


OFFSETS = [("f32", o) for o in (0.0, 100.0, 1e4, -1e4, 1e10, -1e10, 3e38, "lowest")]
OFFSETS += [("bf16", o) for o in (100.0, 1e4, -1e10, "lowest")] + [("f16", o) for o in (100.0, -1e4, "lowest")]


@pytest.mark.parametrize("dtype,offset", OFFSETS)
@pytest.mark.parametrize("n,t,v", [(2, 3, 601), (2, 2, 9001), (2, 300, 130), (2, 260, 4099)])
def test_gradient_of_rows_with_an_offset(n, t, v, dtype, offset):
    x, labels, lab = offset_case(n, t, v, offset, dtype)
    logp, lse = bcl.token_logprob(x, labels)
    assert bool(lse.isfinite().all())
    g = torch.from_numpy(rng(201, n, t).standard_normal((n, t))).to(DEV, torch.float32)
    check_gradient(bcl.token_logprob_bwd(x, labels, lse, g), x, lab, lse, f64(g), dtype)
    r, d = bcl.preference_loss_step(x, labels, logp - 0.1, beta=0.3, kind="ipo", average=True)
    check_gradient(d, x, lab, r.lse, np.repeat(f64(r.slope)[:, None], t, 1), dtype)
    adv = torch.tensor([1.0, -0.5], device=DEV)
    p, d = bcl.policy_loss_step(x, labels, logp, adv, reduction="sum")
    assert bool(p.lse.isfinite().all())
    check_gradient(d, x, lab, p.lse, f64(p.slope), dtype)


@pytest.mark.parametrize("n_pos", [1, 300])  # rows fewer and more than a step's gradient works the slopes out for
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_preference_of_infinite_log_ratios(smoothing, n_pos):
    # pair 0: the chosen label's logit is -inf, z = -inf; pair 1: the rejected one's, z = +inf; pair 2: none
    beta, v = 0.25, 50
    x = torch.zeros(6, n_pos, v, device=DEV)
    lab = torch.full((6, n_pos), 7, dtype=torch.int64, device=DEV)
    x[0, 0, 7] = x[4, 0, 7] = float("-inf")
    ref = torch.zeros(6, n_pos, device=DEV)
    r, d = bcl.preference_loss_step(x, lab, ref, beta=beta, label_smoothing=smoothing)
    f = bcl.preference_loss_fwd(x, lab, ref, beta=beta, label_smoothing=smoothing)
    e = smoothing
    slope = [-beta * (1 - e), beta * e, -beta * (0.5 - e)]  # d loss / d h at z = -inf, +inf and 0
    for got in (r, f):
        loss = f64(got.loss)
        assert loss[0] == np.inf and loss[1] == (np.inf if e else 0.0) and abs(loss[2] - np.log(2.0)) <= 4 * U
        within(f64(got.slope), np.array([*slope, *[-s for s in slope]]), 2 * U)
    assert bool(d.isfinite().all()) and torch.equal(d[0, 0, 7], r.slope[0])
    # the separate backward gives the same
    two = bcl.preference_loss_bwd(x, lab, f.lse, f.slope, torch.ones(3, device=DEV))
    assert torch.equal(two, d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [3, 100, 128, 1000, 1500, 4090, 5001, 16380, 16384])
def test_layer_norm_bwd_of_constant_rows_with_a_large_mean(d, dtype):
    # hat is 0 all along the row; (0 - mean) rstd, what a place past the row's end would give, is past fp32's range
    r = rng(210, d)
    mean = stored(np.array([1e37, -1e37, 3.0]), dtype)[0].to(DEV)
    x = mean[:, None].expand(3, d).contiguous()
    dy, dyr = stored(r.standard_normal((3, d)), dtype)
    w, wr = stored(1.0 + 0.2 * r.standard_normal(d), "f32")
    rstd = torch.full((3,), 316.0, device=DEV)
    dx, dw, db = bcl.layer_norm_bwd(x, w.to(DEV), mean.float(), rstd, dy.to(DEV))
    g = dyr * wr
    want = 316.0 * (g - g.mean(-1, keepdims=True))
    s, tiny = STORE[dtype]
    e = (d / 64 + 24) * U  # a sum's error of its magnitudes, and the other roundings
    within(f64(dx), want, s * np.abs(want) * 1.01 + tiny + 316.0 * e * (np.abs(g) + np.abs(g).mean(-1, keepdims=True)))
    assert not dw.any()
    within(f64(db), dyr.sum(0), 8 * U * np.abs(dyr).sum(0))


def test_policy_step_of_more_rows_than_a_launch_has_threads_for():
    # 2^26 + 5 rows, which at a wave a row is past the 2^32 threads that one launch may have
    t, v = (1 << 26) + 5, 16
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn(1, t, v, generator=g, device=DEV, dtype=torch.bfloat16)
    lab = torch.randint(0, v, (1, t), generator=g, device=DEV)
    lab[0, ::7] = IGNORE
    old = torch.full((1, t), -2.5, device=DEV)
    adv = torch.ones(1, device=DEV)
    r, d = bcl.policy_loss_step(x, lab, old, adv, reduction="token")
    live = lab[0] != IGNORE
    ratio = (r.logp[0].double() - old[0].double()).exp()
    each = -torch.minimum(ratio, ratio.clamp(0.8, 1.2))
    want = float(torch.where(live, each, 0.0).sum() / live.sum())
    within(float(r.loss), want, 4 * U * abs(want))
    at = torch.cat([torch.randint(0, t, (4000,), generator=g, device=DEV), torch.arange(t - 70, t, device=DEV)])
    rows, some = f64(x[0, at]), lab[0, at].cpu().numpy()
    lse = np.log(np.exp(rows).sum(-1))
    on = some != IGNORE
    within(f64(r.lse[0, at]), np.where(on, lse, 0.0), 40 * U * (1 + np.abs(lse)))
    check_gradient(d[0, at], x[0, at], some, r.lse[0, at], f64(r.slope[0, at]), "bf16")
    assert not r.slope[0, ::7].any() and bool(r.slope[0, 1::7].ne(0).any())
