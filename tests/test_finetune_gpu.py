"""GPU parity of the fine-tuning operators against the float64 oracle.

Bounds come from tests/finetune_util.py: the worst case of the kernels' fp32
arithmetic plus one rounding to storage.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import block_circulant_layers_amd as bcl
from oracle import finetune_oracle as fo
from tests import finetune_util as fu
from tests.finetune_util import IGNORE, U, f64, rng, store_err, stored, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = ["f32", "bf16", "f16"]


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def exact32(a):
    """(device float32 tensor, float64 array of its values)."""
    t, ref = stored(a, "f32")
    return t.to(DEV), ref


# ---------------------------------------------------------------------------
# layer normalisation
# ---------------------------------------------------------------------------
def norm_fwd_bounds(x, mean, rstd, w, dtype, y):
    d = x.shape[-1]
    e_mean = fu.sum_err(d) * np.abs(x).mean(-1) + 2 * U * np.abs(mean)
    mid = np.abs(x - mean[..., None])
    # the mean square of x - mean: the mean's error enters squared, the subtractions' at first order
    rel_var = fu.sum_err(d) + 8 * U + (2 * e_mean * mid.mean(-1) + e_mean**2) * rstd**2
    e_rstd = rstd * (rel_var / 2 + 4 * U)
    aw = 1.0 if w is None else np.abs(w)
    e_hat = (e_mean[..., None] + 2 * U * mid) * rstd[..., None] + mid * e_rstd[..., None]
    return store_err(y, dtype) + e_hat * aw + 4 * U * (np.abs(y) + mid * rstd[..., None] * aw), e_mean, e_rstd


SHAPES = [(1, 1), (1, 4096), (3, 2), (5, 7), (2, 63), (7, 64), (4, 65), (33, 257), (3, 1023), (2, 4097), (300, 512),
          (5, 16384), (2, 20000), (1030, 33), (1, 131073)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_layer_norm_fwd(rows, d, dtype):
    r = rng(10, rows, d)
    xt, x = stored(2.0 * r.standard_normal((rows, d)) + 3.0, dtype)
    w, wr = exact32(1.0 + 0.3 * r.standard_normal(d))
    b, br = exact32(r.standard_normal(d))
    for use_w, use_b in ((True, True), (True, False), (False, False), (False, True)):
        want, mean, rstd = fo.layer_norm(x, wr if use_w else None, br if use_b else None, 1e-5)
        y, m, s = bcl.layer_norm_fwd(xt.to(DEV), w if use_w else None, b if use_b else None, 1e-5)
        bound, e_mean, e_rstd = norm_fwd_bounds(x, mean, rstd, wr if use_w else None, dtype, want)
        within(f64(m), mean, e_mean)
        within(f64(s), rstd, e_rstd)
        within(f64(y), want, bound + (4 * U * np.abs(br) if use_b else 0.0))


def norm_bwd_bounds(x, w, mean, rstd, dy, dx, dtype):
    d = x.shape[-1]
    hat = np.abs((x - mean[:, None]) * rstd[:, None])
    g = np.abs(dy * (1.0 if w is None else w))
    e = fu.sum_err(d) + 8 * U
    inner = g + g.mean(-1, keepdims=True) + hat * (g * hat).mean(-1, keepdims=True)
    bdx = store_err(dx, dtype) + rstd[:, None] * (e * inner + 8 * U * inner)
    # a sum over rows is split over at least... no split is assumed: n sequential terms
    n = x.shape[0]
    es = (n + 16) * U
    return bdx, (es + 6 * U) * (np.abs(dy) * hat).sum(0), es * np.abs(dy).sum(0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_layer_norm_bwd(rows, d, dtype):
    r = rng(11, rows, d)
    xt, x = stored(2.0 * r.standard_normal((rows, d)) + 3.0, dtype)
    gt, dy = stored(r.standard_normal((rows, d)), dtype)
    w, wr = exact32(1.0 + 0.3 * r.standard_normal(d))
    _, m0, s0 = fo.layer_norm(x)
    (m, mr), (s, sr) = exact32(m0), exact32(s0)
    xd, gd = xt.to(DEV), gt.to(DEV)
    for use_w in (True, False):
        dx0, dw0, db0 = fo.layer_norm_bwd(x, wr if use_w else None, mr, sr, dy)
        bx, bw, bb = norm_bwd_bounds(x, wr if use_w else None, mr, sr, dy, dx0, dtype)
        dx, dw, db = bcl.layer_norm_bwd(xd, w if use_w else None, m, s, gd)
        within(f64(dx), dx0, bx)
        within(f64(dw), dw0, bw)
        within(f64(db), db0, bb)
    # each output alone, and the gradient in place
    only = bcl.layer_norm_bwd(xd, w, m, s, gd, need_dw=False, need_db=False)
    ref = bcl.layer_norm_bwd(xd, w, m, s, gd)
    assert only[1] is None and only[2] is None and torch.equal(only[0], ref[0])
    for k in ("need_dw", "need_db"):
        part = bcl.layer_norm_bwd(xd, w, m, s, gd, **{"need_dx": False, "need_dw": False, "need_db": False, k: True})
        assert part[0] is None
        i = 1 if k == "need_dw" else 2
        within(f64(part[i]), (dw0, db0)[i - 1], (bw, bb)[i - 1])
    g2 = gd.clone()
    dx, dw, db = bcl.layer_norm_bwd(xd, w, m, s, g2, dx=g2)
    assert dx is g2 and torch.equal(g2, ref[0]) and torch.equal(dw, ref[1]) and torch.equal(db, ref[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 255, 1024])
def test_layer_norm_strided_rows(d, dtype):
    # rows inside a wider buffer at an odd element offset; results equal the contiguous call's bit for bit
    r = rng(12, d)
    wide, _ = stored(r.standard_normal((6, d + 13)), dtype)
    wide = wide.to(DEV)
    for off in (0, 3, 8):
        x = wide[:, off:off + d]
        w = dev(1.0 + 0.1 * r.standard_normal(d))
        y, m, s = bcl.layer_norm_fwd(x, w)
        y0, m0, s0 = bcl.layer_norm_fwd(x.contiguous(), w)
        bound = store_err(f64(y0), dtype) * 2 + 1e-5 * np.abs(f64(y0))
        within(f64(y), f64(y0), bound)
        out = torch.full((6, d + 7), 5.0, dtype=x.dtype, device=DEV)
        bcl.layer_norm_fwd(x, w, y=out[:, 1:1 + d])
        within(f64(out[:, 1:1 + d]), f64(y0), bound)
        assert bool((out[:, 0] == 5.0).all()) and bool((out[:, 1 + d:] == 5.0).all())
        dx, dw, db = bcl.layer_norm_bwd(x, w, m0, s0, x)
        dx0, dw0, db0 = bcl.layer_norm_bwd(x.contiguous(), w, m0, s0, x.contiguous())
        within(f64(dx), f64(dx0), store_err(f64(dx0), dtype) * 2 + 1e-5)
        within(f64(dw), f64(dw0), 1e-4)
        within(f64(db), f64(db0), 1e-4)


def test_layer_norm_constant_rows_and_large_means():
    # a constant row has hat = 0 exactly; a mean of 1e4 with spread 1 keeps its variance
    x = torch.full((2, 300), 7.0, device=DEV)
    y, m, s = bcl.layer_norm_fwd(x, None, None, 1e-5)
    assert torch.equal(y, torch.zeros_like(y)) and bool((m == 7.0).all())
    r = rng(13)
    t, ref = stored(1e4 + r.standard_normal((4, 4096)), "f32")
    want, mean, rstd = fo.layer_norm(ref)
    y, m, s = bcl.layer_norm_fwd(t.to(DEV))
    bound, e_mean, e_rstd = norm_fwd_bounds(ref, mean, rstd, None, "f32", want)
    within(f64(m), mean, e_mean)
    within(f64(s), rstd, e_rstd)
    within(f64(y), want, bound)


def test_layer_norm_non_finite_rows_stay_apart():
    r = rng(14)
    x = dev(r.standard_normal((4, 1000)))
    ref = bcl.layer_norm_fwd(x)[0]
    x[1, 17], x[2, 3] = float("nan"), float("inf")
    y = bcl.layer_norm_fwd(x)[0]
    assert torch.equal(y[0], ref[0]) and torch.equal(y[3], ref[3])
    assert bool(y[1].isnan().all()) and bool(y[2].isnan().all())


def test_layer_norm_empty():
    x = torch.empty(0, 8, device=DEV)
    y, m, s = bcl.layer_norm_fwd(x)
    assert y.shape == (0, 8) and m.shape == (0,) and s.shape == (0,)
    dw = torch.full((8,), float("nan"), device=DEV)
    dx, dw, db = bcl.layer_norm_bwd(x, None, m, s, x, dw=dw)
    assert dx.shape == (0, 8) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_module_gradients(dtype):
    r = rng(15)
    ln = bcl.LayerNorm(96, device=DEV)
    with torch.no_grad():
        ln.weight.copy_(dev(1 + 0.2 * r.standard_normal(96)))
        ln.bias.copy_(dev(r.standard_normal(96)))
    xt, x = stored(r.standard_normal((3, 5, 96)), dtype)
    gt, dy = stored(r.standard_normal((3, 5, 96)), dtype)
    xd = xt.to(DEV).requires_grad_(True)
    y = ln(xd)
    y.backward(gt.to(DEV))
    wr = f64(ln.weight)
    y0, m0, s0 = fo.layer_norm(x, wr, f64(ln.bias))
    dx0, dw0, db0 = fo.layer_norm_bwd(x, wr, m0, s0, dy)
    tol = {"f32": 1e-5, "bf16": 2e-2}[dtype]
    assert y.dtype == xd.dtype and np.linalg.norm(f64(y) - y0) <= tol * np.linalg.norm(y0)
    assert np.linalg.norm(f64(xd.grad).reshape(-1, 96) - dx0) <= tol * np.linalg.norm(dx0)
    assert np.linalg.norm(f64(ln.weight.grad) - dw0) <= 1e-5 * np.linalg.norm(dw0)
    assert np.linalg.norm(f64(ln.bias.grad) - db0) <= 1e-5 * np.linalg.norm(db0)
    # a transposed input, whose rows the kernels cannot address, goes through a copy
    xt2 = xd.detach().transpose(0, 1).transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(ln(xt2), ln(xt2.contiguous()))


# ---------------------------------------------------------------------------
# logits
# ---------------------------------------------------------------------------
LOGITS = [(2, 1, 1), (2, 3, 2), (2, 5, 7), (4, 2, 64), (2, 7, 255), (2, 3, 1000), (6, 4, 1009), (2, 2, 4099),
          (2, 33, 513), (2, 3, 32768), (2, 2, 50001), (2, 1, 131072), (2, 1, 200003), (4, 300, 40)]


def check_logp(logits, lab, logp, lse, lse0, logp0):
    e = np.where(lab != IGNORE, fu.lse_err(logits, lse0), 0.0)
    within(f64(lse), lse0, e)
    within(f64(logp), logp0, e + 2 * U * np.abs(logp0))
    return e


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,t,v", LOGITS)
def test_token_logprob(n, t, v, dtype):
    xt, x, lab = fu.logit_case((20, n, t, v), n, t, v, dtype, empty=(1,) if t > 1 else ())
    logp0, lse0 = fo.token_logprob(x, lab)
    xd, ld = xt.to(DEV), dev(lab, torch.int64)
    logp, lse = bcl.token_logprob(xd, ld)
    check_logp(x, lab, logp, lse, lse0, logp0)
    g, gr = exact32(rng(21, n, t, v).standard_normal((n, t)))
    lse_t, lse_r = exact32(lse0)
    want = fo.logits_grad(x, lab, gr)
    d = bcl.token_logprob_bwd(xd, ld, lse_t, g)
    within(f64(d), want, fu.grad_err(want, x, lab, gr, lse0, dtype))
    assert not f64(d)[lab == IGNORE].any()
    xi = xd.clone()
    assert bcl.token_logprob_bwd(xi, ld, lse_t, g, dlogits=xi) is xi
    assert torch.equal(xi, d)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind,smoothing", [("sigmoid", 0.0), ("sigmoid", 0.1), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("n,t,v", [(2, 1, 9), (2, 40, 333), (6, 17, 1009), (8, 3, 8200)])
def test_preference(n, t, v, kind, smoothing, dtype):
    for average in (False, True):
        xt, x, lab = fu.logit_case((22, n, t, v), n, t, v, dtype, empty=(0,) if n > 2 else ())
        logp0, lse0 = fo.token_logprob(x, lab)
        ref, rr = exact32(logp0 + 0.3 * rng(23, n, t).standard_normal((n, t)))
        kw = dict(beta=0.25, kind=kind, average=average)
        loss0, ratio0, slope0 = fo.preference(logp0, lab, rr, 0.25, kind, smoothing, average)
        xd, ld = xt.to(DEV), dev(lab, torch.int64)
        r, d = bcl.preference_loss_step(xd, ld, ref, label_smoothing=smoothing, scale=0.5, **kw)
        e = check_logp(x, lab, r.logp, r.lse, lse0, logp0) + 2 * U * np.abs(logp0)
        count = np.maximum(1, (lab != IGNORE).sum(1)) if average else 1.0
        e_ratio = e.sum(1) / count + 4 * U * np.abs(ratio0)
        within(f64(r.logratio), ratio0, e_ratio)
        e_h = e_ratio[: n // 2] + e_ratio[n // 2:]
        h = ratio0[: n // 2] - ratio0[n // 2:]
        first = {"sigmoid": 0.25, "hinge": 0.25}.get(kind, 2 * np.abs(h - 2.0) + e_h)  # |d loss / d h|
        second = {"sigmoid": 0.25**2 / 4, "hinge": 0.0}.get(kind, 2.0)
        within(f64(r.loss), loss0, first * e_h + 8 * U * (np.abs(loss0) + 1e-3))
        e_slope = np.tile(second * e_h, 2) / count + 8 * U * np.abs(slope0)
        if kind == "hinge":  # the slope jumps where the margin is met: only away from it
            assert (np.abs(1 - 0.25 * h) > 0.25 * e_h).all()
        within(f64(r.slope), slope0, e_slope)
        g = np.broadcast_to(0.5 * slope0[:, None], lab.shape)
        want = fo.logits_grad(x, lab, g)
        bound = fu.grad_err(want, x, lab, g, lse0, dtype) + 0.5 * e_slope[:, None, None]
        within(f64(d), want, bound)
        assert not f64(d)[lab == IGNORE].any()
        # the separate calls give what the step gave
        f = bcl.preference_loss_fwd(xd, ld, ref, label_smoothing=smoothing, **kw)
        for a, b in zip(f, r):
            within(f64(a), f64(b), 1e-5 * (1 + np.abs(f64(b))))
        d2 = bcl.preference_loss_bwd(xd, ld, r.lse, r.slope, torch.full((n // 2,), 0.5, device=DEV))
        within(f64(d2), f64(d), fu.grad_err(want, x, lab, g, lse0, dtype) * 2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("n,t,v", [(1, 1, 5), (3, 40, 333), (5, 17, 1009), (2, 3, 8200), (2, 2, 70001), (600, 2, 50)])
def test_policy(n, t, v, reduction, dtype):
    xt, x, lab = fu.logit_case((24, n, t, v), n, t, v, dtype, masked=0.0 if n == 1 else 0.3,
                               empty=(n - 1,) if n > 1 else ())
    logp0, lse0 = fo.token_logprob(x, lab)
    r0 = rng(25, n, t, v)
    old, oldr = exact32(logp0 + 0.3 * r0.standard_normal((n, t)))
    ref, refr = exact32(logp0 + 0.3 * r0.standard_normal((n, t)))
    for per_token, with_ref in ((False, True), (True, False)):
        adv, advr = exact32(r0.standard_normal((n, t) if per_token else (n, 1)))
        kw = dict(clip_low=0.1, clip_high=0.25, kl_coef=0.2, reduction=reduction)
        loss0, kl0, slope0 = fo.policy(logp0, lab, oldr, advr, refr if with_ref else None, 0.1, 0.25, 0.2, reduction)
        xd, ld = xt.to(DEV), dev(lab, torch.int64)
        r, d = bcl.policy_loss_step(xd, ld, old, adv, ref_logp=ref if with_ref else None, scale=2.0, **kw)
        e = check_logp(x, lab, r.logp, r.lse, lse0, logp0) + 2 * U * np.abs(logp0)
        live = lab != IGNORE
        ratio = np.exp(np.where(live, logp0 - oldr, 0.0))
        a = np.broadcast_to(np.abs(advr), lab.shape)
        if reduction == "token":
            w = live / max(1, live.sum())
        elif reduction == "sequence":
            w = live / np.maximum(1, live.sum(1, keepdims=True)) / n
        else:
            w = live * 1.0
        # the clipped range's ends, where the slope jumps, are not within the error of any ratio
        far = np.minimum(np.abs(ratio - 0.9), np.abs(ratio - 1.25)) > 2 * ratio * e + 1e-12
        assert far[live].all()
        q = np.abs(np.expm1(np.where(live, refr - logp0, 0.0))) if with_ref else np.zeros(lab.shape)
        e_term = (ratio * a + 0.2 * q) * (e + 4 * U) * 1.1 + 0.2 * e**2
        within(f64(r.loss), loss0, (w * e_term).sum() + 8 * U * (np.abs(loss0) + 1e-4))
        within(f64(r.kl), kl0, (w * (q * e + e**2)).sum() * 1.1 + 8 * U * (kl0 + 1e-6))
        e_slope = w * (ratio * a + 0.2 * (q + 1.0)) * (e + 4 * U) * 1.2 + 4 * U * np.abs(slope0)
        within(f64(r.slope), slope0, e_slope)
        g = 2.0 * slope0
        want = fo.logits_grad(x, lab, g)
        within(f64(d), want, fu.grad_err(want, x, lab, g, lse0, dtype) + 2 * e_slope[..., None])
        assert not f64(d)[~live].any()
        f = bcl.policy_loss_fwd(xd, ld, old, adv, ref_logp=ref if with_ref else None, **kw)
        for p, s in zip(f, r):
            within(f64(p), f64(s), 1e-5 * (1 + np.abs(f64(s))))
        d2 = bcl.policy_loss_bwd(xd, ld, r.lse, r.slope, torch.full((), 2.0, device=DEV))
        within(f64(d2), f64(d), fu.grad_err(want, x, lab, g, lse0, dtype) * 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_strided(dtype):
    # positions of a longer sequence, a slice of a wider vocabulary axis at an odd offset, and time-major logits
    n, t, v = 4, 6, 1003
    xt, x, lab = fu.logit_case((26,), n, t + 1, v + 10, dtype, masked=0.2)
    full = xt.to(DEV)
    lab = np.where(lab == IGNORE, IGNORE, np.minimum(lab, v - 1))[:, 1:]
    ld = dev(lab, torch.int64)
    for view in (full[:, :-1, 5:5 + v], full[:, :-1, :v], full[:, 1:, 8:8 + v],
                 full[:, :-1, :v].transpose(0, 1).contiguous().transpose(0, 1)):
        ref = f64(view)
        logp0, lse0 = fo.token_logprob(ref, lab)
        logp, lse = bcl.token_logprob(view, ld)
        check_logp(ref, lab, logp, lse, lse0, logp0)
        g, gr = exact32(rng(27).standard_normal((n, t)))
        want = fo.logits_grad(ref, lab, gr)
        bound = fu.grad_err(want, ref, lab, gr, lse0, dtype)
        within(f64(bcl.token_logprob_bwd(view, ld, lse, g)), want, bound)
        # into a strided buffer whose other elements stay
        out = torch.full((n, t + 2, v + 3), 7.0, dtype=full.dtype, device=DEV)
        bcl.token_logprob_bwd(view, ld, lse, g, dlogits=out[:, 1:-1, 1:1 + v])
        within(f64(out[:, 1:-1, 1:1 + v]), want, bound)
        out[:, 1:-1, 1:1 + v] = 7.0
        assert bool((out == 7.0).all())
        # in place in the view: what is outside it stays
        keep = full.clone()
        buf = full.clone()
        inner = buf.as_strided(view.shape, view.stride(), view.storage_offset()) if view._base is full else None
        if inner is not None:
            bcl.token_logprob_bwd(inner, ld, lse, g, dlogits=inner)
            within(f64(inner), want, bound)
            inner.copy_(keep.as_strided(view.shape, view.stride(), view.storage_offset()))
            assert torch.equal(buf, keep)


def test_masked_positions_are_not_read():
    # infinities and NaN at masked positions change nothing, bit for bit
    n, t, v = 4, 5, 777
    xt, x, lab = fu.logit_case((28,), n, t, v, "bf16", masked=0.4, empty=(3,))
    ld = dev(lab, torch.int64)
    xd = xt.to(DEV)
    bad = xd.clone()
    mask = dev(lab == IGNORE, torch.bool)
    bad[mask] = float("nan")
    bad[:, :, ::3][mask] = float("inf")
    old = dev(rng(29).standard_normal((n, t)) - 5.0)
    old_bad = old.clone()
    old_bad[mask] = float("nan")
    adv = torch.ones(n, device=DEV)
    a = bcl.policy_loss_step(xd, ld, old, adv, ref_logp=old, kl_coef=0.1)
    b = bcl.policy_loss_step(bad, ld, old_bad, adv, ref_logp=old_bad, kl_coef=0.1)
    for p, q in zip([*a[0], a[1]], [*b[0], b[1]]):
        assert torch.equal(p, q)
    a = bcl.preference_loss_step(xd, ld, old)
    b = bcl.preference_loss_step(bad, ld, old_bad)
    for p, q in zip([*a[0], a[1]], [*b[0], b[1]]):
        assert torch.equal(p, q)


def test_non_finite_logits_follow_the_formula():
    v = 600
    x = torch.zeros(2, 6, v, device=DEV)
    x[0, 0, 100:] = float("-inf")  # part of the vocabulary excluded
    x[0, 1, :] = float("-inf")  # nothing left: no softmax
    x[0, 2, 5] = float("inf")
    x[0, 3, 7] = float("nan")
    x[0, 4, :] = torch.finfo(torch.float32).min  # the type's lowest value everywhere: uniform
    x[0, 5, 1:] = torch.finfo(torch.float32).min
    lab = torch.zeros(2, 6, dtype=torch.int64, device=DEV)
    logp, lse = bcl.token_logprob(x, lab)
    got = logp[0].tolist()
    assert abs(got[0] + np.log(100)) < 1e-5 and all(np.isnan(got[1:4])) and got[5] == 0.0
    assert abs(got[4]) <= 2.0**104  # the lowest value swallows log v: logp is a rounding of it
    d = bcl.token_logprob_bwd(x, lab, lse, torch.ones_like(logp))
    assert not d[0, 0, 100:].any() and abs(float(d[0, 0, 0]) - 0.99) < 1e-5
    assert bool(d[0, 1:4].isnan().all()) and bool(d[1].isfinite().all())


def test_labels_out_of_range_give_nan_and_touch_nothing_else():
    n, t, v = 2, 4, 130
    xt, x, lab = fu.logit_case((30,), n, t, v, "f32", masked=0.0)
    xd = xt.to(DEV)
    good = bcl.token_logprob(xd, dev(lab, torch.int64))[0]
    lab2 = lab.copy()
    lab2[0, 1], lab2[1, 2], lab2[1, 3] = v, -1, 1 << 40
    ld = dev(lab2, torch.int64)
    logp, lse = bcl.token_logprob(xd, ld)
    hit = lab2 != lab
    assert np.isnan(f64(logp)[hit]).all() and np.array_equal(f64(logp)[~hit], f64(good)[~hit])
    d = bcl.token_logprob_bwd(xd, ld, lse, torch.ones_like(lse))
    assert np.isnan(f64(d)[hit]).all() and np.isfinite(f64(d)[~hit]).all()
    assert np.isnan(f64(bcl.policy_loss_fwd(xd, ld, good, torch.ones(n, device=DEV)).loss))


@pytest.mark.parametrize("n,t", [(2, 0), (0, 3), (0, 0)])
def test_no_positions(n, t):
    x = torch.empty(n, t, 50, device=DEV)
    lab = torch.empty(n, t, dtype=torch.int64, device=DEV)
    e = torch.empty(n, t, device=DEV)
    r, d = bcl.preference_loss_step(x, lab, e, beta=0.5)
    assert d.shape == x.shape and r.loss.shape == (n // 2,)
    assert np.allclose(f64(r.loss), np.log(2.0)) and not r.logratio.any()
    p, d = bcl.policy_loss_step(x, lab, e, torch.empty(n, device=DEV))
    assert float(p.loss) == 0.0 and float(p.kl) == 0.0 and d.shape == x.shape


def test_all_positions_masked():
    x = torch.randn(4, 3, 500, device=DEV)
    lab = torch.full((4, 3), IGNORE, dtype=torch.int64, device=DEV)
    ref = torch.randn(4, 3, device=DEV)
    for average in (False, True):
        r, d = bcl.preference_loss_step(x, lab, ref, average=average)
        assert np.allclose(f64(r.loss), np.log(2.0)) and not r.logratio.any() and not d.any()
    for reduction in ("token", "sequence", "sum"):
        p, d = bcl.policy_loss_step(x, lab, ref, torch.randn(4, device=DEV), ref_logp=ref, reduction=reduction)
        assert float(p.loss) == 0.0 and float(p.kl) == 0.0 and not d.any() and not p.slope.any()


def test_rows_past_32_bit_offsets():
    # the last rows of a bfloat16 batch start past element 2^31
    n, t, v = 2, 33000, 32768
    x = torch.empty(n, t, v, dtype=torch.bfloat16, device=DEV)
    lab = torch.full((n, t), IGNORE, dtype=torch.int64, device=DEV)
    xt, xr, lr = fu.logit_case((31,), 1, 3, v, "bf16", masked=0.0)
    x[1, -3:] = xt[0].to(DEV)
    lab[1, -3:] = dev(lr[0], torch.int64)
    assert (2 * t - 3) * v > 2**31
    logp0, lse0 = fo.token_logprob(xr, lr)
    logp, lse = bcl.token_logprob(x, lab)
    check_logp(xr, lr, logp[1:, -3:], lse[1:, -3:], lse0, logp0)
    g = torch.zeros_like(logp)
    g[1, -3:] = 1.0
    bcl.token_logprob_bwd(x, lab, lse, g, dlogits=x)
    want = fo.logits_grad(xr, lr, np.ones((1, 3)))
    within(f64(x[1:, -3:]), want, fu.grad_err(want, xr, lr, np.ones((1, 3)), lse0, "bf16"))
    assert not bool(x[1, -5:-3].any())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("inplace", [False, True])
def test_autograd_losses(inplace, dtype):
    n, t, v = 4, 6, 301
    xt, x, lab = fu.logit_case((32,), n, t, v, dtype, masked=0.2)
    ld = dev(lab, torch.int64)
    logp0, lse0 = fo.token_logprob(x, lab)
    r0 = rng(33)
    ref, refr = exact32(logp0 + 0.2 * r0.standard_normal((n, t)))
    up, upr = exact32(r0.standard_normal(n // 2))
    adv, advr = exact32(r0.standard_normal(n))

    def leaf():
        base = xt.to(DEV).requires_grad_(True)
        return base, base * 1.0  # logits that autograd made, as a model's head does

    base, z = leaf()
    loss, ratio = bcl.preference_loss(z, ld, ref, beta=0.2, label_smoothing=0.1, inplace=inplace)
    assert not ratio.requires_grad
    (loss * up).sum().backward()
    slope = fo.preference(logp0, lab, refr, 0.2, "sigmoid", 0.1)[2]
    g = np.tile(upr, 2)[:, None] * slope[:, None] * np.ones(lab.shape)
    want = fo.logits_grad(x, lab, g)
    tol = {"f32": 1e-5, "f16": 1e-3}[dtype]
    assert np.linalg.norm(f64(base.grad) - want) <= tol * np.linalg.norm(want)
    base, z = leaf()
    loss, kl = bcl.policy_loss(z, ld, ref, adv, ref_logp=ref, kl_coef=0.1, inplace=inplace)
    (3.0 * loss).backward()
    want = fo.logits_grad(x, lab, 3.0 * fo.policy(logp0, lab, refr, advr[:, None], refr, kl_coef=0.1)[2])
    assert np.linalg.norm(f64(base.grad) - want) <= tol * np.linalg.norm(want)
    base, z = leaf()
    bcl.token_logp(z, ld, inplace=inplace).sum().backward()
    want = fo.logits_grad(x, lab, np.ones(lab.shape))
    assert np.linalg.norm(f64(base.grad) - want) <= tol * np.linalg.norm(want)


def test_policy_gradient_against_differences():
    # the fp32 loss itself moved along the gradient: a central difference of the computed loss
    n, t, v = 3, 4, 97
    xt, x, lab = fu.logit_case((34,), n, t, v, "f32", masked=0.2)
    ld = dev(lab, torch.int64)
    logp0, _ = fo.token_logprob(x, lab)
    old = dev(logp0 + 0.05 * rng(35).standard_normal((n, t)))
    adv = dev(np.array([1.0, -0.5, 2.0]))
    xd = xt.to(DEV)
    kw = dict(ref_logp=old, kl_coef=0.3, reduction="sum")
    _, d = bcl.policy_loss_step(xd, ld, old, adv, **kw)
    step = d / d.norm()
    h = 1e-2
    up = bcl.policy_loss_fwd(xd + h * step, ld, old, adv, **kw).loss.double()
    down = bcl.policy_loss_fwd(xd - h * step, ld, old, adv, **kw).loss.double()
    slope = float((up - down) / (2 * h))
    # truncation h^2 f''' / 6 with f''' of the order of the gradient, rounding 1e-6 f / h
    assert abs(slope - float(d.norm())) <= 2e-3 * float(d.norm())


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------
def tensors(key, shapes, dtypes):
    r = rng(*key)
    got = [stored(r.standard_normal(s) * 10.0 ** r.integers(-3, 2), dt) for s, dt in zip(shapes, dtypes)]
    return [t.to(DEV) for t, _ in got], [a for _, a in got]


CLIPS = [
    ([(1,)], ["f32"]),
    ([(7,), (0,), (3, 5)], ["f32", "bf16", "f16"]),
    ([(16384,)] * 9, ["f32"] * 9),
    ([(16385,), (1,), (70001,), (16383,)], ["bf16", "f32", "f16", "f32"]),
    ([(k,) for k in range(260)], [("f32", "bf16", "f16")[k % 3] for k in range(260)]),
    ([(3, 100003)], ["bf16"]),
    ([(1 << 22,), (5,)], ["f32", "f16"]),
]


@pytest.mark.parametrize("case", range(len(CLIPS)))
@pytest.mark.parametrize("max_norm", [0.0, 0.37, 1e12])
def test_clip(case, max_norm):
    shapes, dtypes = CLIPS[case]
    ts, refs = tensors((40, case), shapes, dtypes)
    norm0, want = fo.clip(refs, max_norm)
    e_norm = 4 * U * norm0
    within(f64(bcl.grad_norm(ts)), norm0, e_norm)
    out = [torch.full_like(t, float("nan")) for t in ts]
    before = [t.clone() for t in ts]
    norm = bcl.clip_grad_norm(ts, max_norm, out=out)
    within(f64(norm), norm0, e_norm)
    for t, b in zip(ts, before):
        assert torch.equal(t, b)
    for o, w, dt in zip(out, want, dtypes):
        within(f64(o), w, store_err(w, dt) + 4 * U * np.abs(w))
    norm2 = bcl.clip_grad_norm(ts, max_norm)  # in place
    assert torch.equal(norm2, norm)
    for t, o in zip(ts, out):
        assert torch.equal(t, o)


def test_clip_packed_bucket_and_odd_offsets():
    # tensors packed one after another in one buffer, at any element boundary, clipped into another such buffer
    r = rng(41)
    sizes = [1, 2, 3, 5, 1000, 40001, 7, 16384, 9]
    for dt in ("f32", "bf16", "f16"):
        flat, ref = stored(r.standard_normal(sum(sizes) + 3), dt)
        flat = flat.to(DEV)
        out = torch.full((len(flat) + 5,), 9.0, dtype=flat.dtype, device=DEV)
        for lead in (0, 1, 4):
            at, gs, os_ = 0, [], []
            for s in sizes:
                gs.append(flat[at:at + s])
                os_.append(out[lead + at:lead + at + s])
                at += s
            norm = bcl.clip_grad_norm(gs, 1.0, out=os_)
            n0, want = fo.clip([ref[:at]], 1.0)
            within(f64(norm), n0, 4 * U * n0)
            within(f64(out[lead:lead + at]), want[0], store_err(want[0], dt) + 4 * U * np.abs(want[0]))
            assert bool((out[:lead] == 9.0).all()) and bool((out[lead + at:] == 9.0).all())
            out.fill_(9.0)


def test_clip_extreme_values():
    # squares past fp32's range on both sides, and values that are not finite
    big = torch.full((1000,), 1e30, device=DEV)
    n = bcl.clip_grad_norm([big], 1.0)
    within(float(n), 1e30 * np.sqrt(1000.0), 1e30 * 1e-5)
    within(f64(big), np.full(1000, 1 / np.sqrt(1000.0)), 1e-6)
    tiny = torch.full((1000,), 1e-30, device=DEV)
    within(float(bcl.grad_norm([tiny])), 1e-30 * np.sqrt(1000.0), 1e-35)
    for bad in (float("inf"), float("nan")):
        a, b = torch.ones(10, device=DEV), torch.ones(5, device=DEV)
        b[2] = bad
        n = bcl.clip_grad_norm([a, b], 1.0)
        assert not bool(n.isfinite())
        if bad == float("inf"):  # the factor is 0
            assert not a.any() and bool(b[2].isnan()) and not b[:2].any()
        else:
            assert bool(a.isnan().all()) and bool(b.isnan().all())


def test_clip_parameters():
    layer = bcl.BlockCirculantLinear(64, 64, 16, device=DEV)
    ln = bcl.LayerNorm(64, device=DEV)
    layer(ln(torch.randn(8, 64, device=DEV))).square().sum().backward()
    params = [*layer.parameters(), *ln.parameters(), torch.nn.Parameter(torch.ones(3, device=DEV))]
    refs = [f64(p.grad) for p in params[:-1]]
    n0, want = fo.clip(refs, 0.5)
    n = bcl.clip_grad_norm_(params, 0.5)
    within(float(n), n0, 4 * U * n0)
    for p, w in zip(params, want):
        within(f64(p.grad), w, 4 * U * np.abs(w) + 1e-45)
    # a gradient whose axes are permuted is one block of memory all the same
    g = torch.randn(5, 7, device=DEV).t()
    r = f64(g)
    bcl.clip_grad_norm([g], 0.1)
    within(f64(g), fo.clip([r], 0.1)[1][0], 1e-6)
    assert float(bcl.clip_grad_norm_([torch.nn.Parameter(torch.ones(2, device=DEV))], 1.0)) == 0.0


# ---------------------------------------------------------------------------
# streams, graphs, repeatability
# ---------------------------------------------------------------------------
def _everything(x, w, dy, logits, lab, ref, adv, grads, out):
    y, m, s = bcl.layer_norm_fwd(x, w, None)
    res = [y, m, s, *bcl.layer_norm_bwd(x, w, m, s, dy)]
    r, d = bcl.preference_loss_step(logits, lab, ref)
    res += [*r, d]
    p, d = bcl.policy_loss_step(logits, lab, ref, adv, ref_logp=ref, kl_coef=0.1)
    res += [*p, d]
    res += [*bcl.token_logprob(logits, lab), bcl.clip_grad_norm(grads, 1.0, out=out), *out]
    return res


def _inputs():
    r = rng(50)
    x, dy = (stored(r.standard_normal((37, 520)), "bf16")[0].to(DEV) for _ in range(2))
    xt, _, lab = fu.logit_case((51,), 4, 9, 5003, "bf16", masked=0.3)
    ref = dev(r.standard_normal((4, 9)) - 6.0)
    grads = [dev(r.standard_normal(k)) for k in (5, 70000, 333)]
    return (x, dev(1 + 0.1 * r.standard_normal(520)), dy, xt.to(DEV), dev(lab, torch.int64), ref,
            dev(r.standard_normal(4)), grads, [torch.empty_like(g) for g in grads])


def test_results_repeat_bitwise():
    args = _inputs()
    first = [t.clone() for t in _everything(*args)]
    for _ in range(5):
        for a, b in zip(first, _everything(*args)):
            assert torch.equal(a, b)


def test_graph_replays():
    args = _inputs()
    eager = [t.clone() for t in _everything(*args)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _everything(*args)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = _everything(*args)
    for i in range(4):
        for t in res:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(eager, res)):
            assert torch.equal(a, b), (i, k)


def test_another_stream():
    # the `stream` argument: work and workspaces on that stream, while the current one runs other work
    x, w, dy, logits, lab, ref, adv, grads, out = _inputs()
    want = [t.clone() for t in _everything(x, w, dy, logits, lab, ref, adv, grads, out)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        got = []
        for _ in range(3):
            y, m, rs = bcl.layer_norm_fwd(x, w, None, stream=s)
            got = [y, m, rs, *bcl.layer_norm_bwd(x, w, m, rs, dy, stream=s)]
            r, d = bcl.preference_loss_step(logits, lab, ref, stream=s)
            got += [*r, d]
            p, d = bcl.policy_loss_step(logits, lab, ref, adv, ref_logp=ref, kl_coef=0.1, stream=s)
            got += [*p, d]
            got += [*bcl.token_logprob(logits, lab, stream=s), bcl.clip_grad_norm(grads, 1.0, out=out, stream=s), *out]
            junk = torch.full((1 << 20,), float("nan"), device=DEV)  # noqa: F841  takes freed blocks of its own stream
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,v", [("f32", 5003), ("bf16", 4099), ("f16", 16390), ("bf16", 50001), ("f32", 33001),
                                     ("bf16", 131072), ("f16", 140001)])
def test_policy_step_many_rows(v, dtype):
    # enough rows that a step holds them in registers: a wave a row, and workgroups of 256 to 1024 threads, and a
    # row past the widest; few unmasked rows keep the oracle quick
    n, t = 8, 130
    r0 = rng(60, v)
    lab = np.full((n, t), IGNORE)
    live = r0.choice(n * t, size=24, replace=False)
    lab.reshape(-1)[live] = r0.integers(0, v, size=24)
    lab = lab.astype(np.int64)
    g = torch.Generator(device=DEV).manual_seed(v)
    xd = torch.randn(n, t, v, generator=g, device=DEV).mul_(3.0).to(fu.TORCH[dtype])
    rows = f64(xd.reshape(n * t, v)[torch.from_numpy(live).to(DEV)])  # the unmasked rows alone, one sequence each
    small = lab.reshape(-1)[live][:, None]
    logp0, lse0 = fo.token_logprob(rows[:, None], small)
    old, oldr = exact32(logp0 + 0.2 * r0.standard_normal(logp0.shape))
    adv, advr = exact32(r0.standard_normal(logp0.shape))
    _, _, slope0 = fo.policy(logp0, small, oldr, advr, reduction="token")
    full_old = torch.zeros(n * t, device=DEV)
    full_adv = torch.zeros(n * t, device=DEV)
    at = torch.from_numpy(live).to(DEV)
    full_old[at], full_adv[at] = old[:, 0], adv[:, 0]
    r, d = bcl.policy_loss_step(xd, dev(lab, torch.int64), full_old.view(n, t), full_adv.view(n, t))
    e = fu.lse_err(rows[:, None], lse0) + 2 * U * np.abs(logp0)
    within(f64(r.logp.reshape(-1)[at])[:, None], logp0, e)
    e_slope = np.abs(slope0) * (e + 4 * U) * 1.2 + 4 * U * np.abs(slope0)
    within(f64(r.slope.reshape(-1)[at])[:, None], slope0, e_slope)
    want = fo.logits_grad(rows[:, None], small, slope0)
    got = f64(d.reshape(n * t, v)[at])[:, None]
    within(got, want, fu.grad_err(want, rows[:, None], small, slope0, lse0, dtype) + e_slope[..., None])
    d.reshape(n * t, v)[at] = 0
    assert not d.any()
    f = bcl.policy_loss_fwd(xd, dev(lab, torch.int64), full_old.view(n, t), full_adv.view(n, t))
    within(f64(f.loss), f64(r.loss), 1e-6)
    # in place
    first = bcl.policy_loss_step(xd, dev(lab, torch.int64), full_old.view(n, t), full_adv.view(n, t))[1]
    bcl.policy_loss_step(xd, dev(lab, torch.int64), full_old.view(n, t), full_adv.view(n, t), dlogits=xd)
    assert torch.equal(xd, first)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,t,v", [(2, 1, 131073), (2, 3, 70001), (4, 60, 9000), (6, 5, 300), (200, 2, 130), (2, 400, 517),
                                   (2, 255, 4099), (2, 256, 4099)])
def test_steps_in_place_equal_steps_apart(n, t, v, dtype):
    # the gradient over the logits themselves: rows in parts, whole rows, either side of the row count that
    # changes the kernels; equal to the gradient beside them and, up to rounding, to the separate calls
    xt, x, lab = fu.logit_case((70, n, t, v), n, t, v, dtype, masked=0.3, empty=(1,) if n > 2 else ())
    xd, ld = xt.to(DEV), dev(lab, torch.int64)
    r0 = rng(71, n, t)
    ref = dev(r0.standard_normal((n, t)) - np.log(v))
    adv = dev(r0.standard_normal(n))
    logp0, lse0 = fo.token_logprob(x, lab)
    for kind in ("sigmoid", "ipo"):
        a, d = bcl.preference_loss_step(xd, ld, ref, kind=kind, average=True)
        buf = xd.clone()
        b, e = bcl.preference_loss_step(buf, ld, ref, kind=kind, average=True, dlogits=buf)
        assert e is buf and torch.equal(d, buf) and all(torch.equal(p, q) for p, q in zip(a, b))
        f = bcl.preference_loss_fwd(xd, ld, ref, kind=kind, average=True)
        assert all(torch.equal(p, q) for p, q in zip(a, f))
    for reduction in ("token", "sequence", "sum"):
        kw = dict(ref_logp=ref, kl_coef=0.1, reduction=reduction)
        a, d = bcl.policy_loss_step(xd, ld, ref, adv, **kw)
        buf = xd.clone()
        b, e = bcl.policy_loss_step(buf, ld, ref, adv, dlogits=buf, **kw)
        assert e is buf and torch.equal(d, buf) and all(torch.equal(p, q) for p, q in zip(a, b))
        check_logp(x, lab, a.logp, a.lse, lse0, logp0)
        f = bcl.policy_loss_fwd(xd, ld, ref, adv, **kw)
        for p, q in zip(a, f):
            within(f64(p), f64(q), 1e-5 * (1 + np.abs(f64(q))))
        want = fo.logits_grad(x, lab, f64(a.slope))
        within(f64(d), fu.representable(want, dtype), fu.grad_err(want, x, lab, f64(a.slope), lse0, dtype) * 1.5)


@pytest.mark.parametrize("dtype,v", [("f32", 2051), ("f16", 4099), ("bf16", 8192), ("bf16", 8199)])
@pytest.mark.parametrize("t", [2047, 2048])
def test_many_rows_either_side_of_a_wave_a_row(t, v, dtype):
    # rows enough that one wave takes a row of up to 16 pieces a lane, and one row a sequence fewer
    n = 2
    xt, x, lab = fu.logit_case((80, t, v), n, t, v, dtype, masked=0.9)
    xd, ld = xt.to(DEV), dev(lab, torch.int64)
    logp0, lse0 = fo.token_logprob(x, lab)
    logp, lse = bcl.token_logprob(xd, ld)
    check_logp(x, lab, logp, lse, lse0, logp0)
    ref = dev(np.where(lab != IGNORE, logp0 + 0.1, 0.0))
    r, d = bcl.preference_loss_step(xd, ld, ref, kind="ipo", average=True)
    assert torch.equal(r.logp, logp) and torch.equal(r.lse, lse)
    g = np.broadcast_to(f64(r.slope)[:, None], lab.shape)
    want = fo.logits_grad(x, lab, g)
    within(f64(d), fu.representable(want, dtype), fu.grad_err(want, x, lab, g, lse0, dtype) * 1.5)
    buf = xd.clone()
    bcl.preference_loss_step(buf, ld, ref, kind="ipo", average=True, dlogits=buf)
    assert torch.equal(buf, d)


@pytest.mark.parametrize("n", [156, 157, 232, 233, 320])
def test_clip_either_side_of_a_table(n):
    sizes = [1 + 37 * k % 211 for k in range(n)]
    dtypes = [("f32", "bf16", "f16")[k % 3] for k in range(n)]
    ts, refs = tensors((90, n), [(s,) for s in sizes], dtypes)
    norm0, want = fo.clip(refs, 0.5)
    out = [torch.full_like(t, float("nan")) if k % 2 else t.clone() for k, t in enumerate(ts)]
    norm = bcl.clip_grad_norm(ts, 0.5, out=out)
    within(f64(norm), norm0, 4 * U * norm0)
    for o, w, dt in zip(out, want, dtypes):
        within(f64(o), w, store_err(w, dt) + 4 * U * np.abs(w))
    some = [t.clone() if k % 2 else t for k, t in enumerate(ts)]  # in place among others elsewhere
    to = [o if k % 2 else torch.empty_like(o) for k, o in enumerate(some)]
    assert torch.equal(bcl.clip_grad_norm(some, 0.5, out=to), norm)
    assert torch.equal(bcl.clip_grad_norm(ts, 0.5), norm)
    for t, o, p in zip(ts, out, to):
        assert torch.equal(t, o) and torch.equal(p, o)


def test_clip_a_tensor_past_one_entry():
    # 1.07 GB of bf16, an odd element in: several entries of the table, chunks on lines throughout
    n = (1 << 29) + 11
    g = torch.Generator(device=DEV).manual_seed(91)
    buf = torch.randn(n + 1, generator=g, device=DEV, dtype=torch.bfloat16)
    t = buf[1:]
    total = sum(float(t[a: a + (1 << 26)].double().square().sum()) for a in range(0, n, 1 << 26))
    first = buf[:1].clone()
    out = torch.empty_like(t)
    norm = bcl.clip_grad_norm([t], 100.0, out=[out])
    within(f64(norm), np.sqrt(total), 4 * U * np.sqrt(total))
    f = min(1.0, 100.0 / (np.sqrt(total) + 1e-6))
    for a in range(0, n, 1 << 26):
        w = t[a: a + (1 << 26)].double() * f
        # a bfloat16 rounding (2^-8) and the factor's and the product's in 24 bits; the least subnormal's half
        assert bool(((out[a: a + (1 << 26)].double() - w).abs() <= (2.0**-8 + 4 * U) * w.abs() + 2.0**-134).all())
    bcl.clip_grad_norm([t], 100.0)
    assert torch.equal(t, out) and torch.equal(buf[:1], first)
