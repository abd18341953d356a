"""GPU tests of layer normalisation with more rows than a launch's workgroups
hold at once: every workgroup takes several rounds, the last of them not by all
its groups, for every number of threads a row; and past the size from which
rows go past the caches.

The 64-bit reference runs on the GPU; bounds are the worst cases of
tests/finetune_util.py, a sum over n rows taken as n sequential additions.
"""

from __future__ import annotations

import pytest
import torch

import block_circulant_layers_amd as bcl
from tests.finetune_util import STORE, TORCH, U, sum_err

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5

# a launch has at most 2048 workgroups forward and 256 or 512 backward, each of 256 threads or one row's
ROUNDS = [(70001, 37), (40003, 250), (20001, 500), (9999, 1000), (5000, 2000), (5001, 1999), (2500, 4093), (2600, 4096),
          (1100, 8192), (1030, 8190), (600, 16383), (520, 16384), (70, 20000)]
LARGE = [(20500, 2048, "f32"), (44000, 4096, "bf16"), (30001, 5999, "f16"), (5200, 16383, "f32")]


def _check(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


def _store(want, dtype):
    s, tiny = STORE[dtype]
    return s * want.abs() * 1.01 + tiny


def _run(rows, d, dtype):
    g = torch.Generator(device=DEV).manual_seed(rows + d)
    x = torch.randn(rows, d, generator=g, device=DEV).mul_(2.0).add_(3.0).to(TORCH[dtype])
    dy = torch.randn(rows, d, generator=g, device=DEV).to(TORCH[dtype])
    w = torch.randn(d, generator=g, device=DEV).mul_(0.3).add_(1.0)
    b = torch.randn(d, generator=g, device=DEV)
    y, mean, rstd = bcl.layer_norm_fwd(x, w, b, EPS)
    xd, wd = x.double(), w.double()
    m = xd.mean(-1)
    mid = xd - m[:, None]
    r = (mid.square().mean(-1) + EPS).rsqrt()
    e_mean = sum_err(d) * xd.abs().mean(-1) + 2 * U * m.abs()
    rel_var = sum_err(d) + 8 * U + (2 * e_mean * mid.abs().mean(-1) + e_mean**2) * r**2
    e_rstd = r * (rel_var / 2 + 4 * U)
    _check(mean, m, e_mean, "mean")
    _check(rstd, r, e_rstd, "rstd")
    hat = mid * r[:, None]
    want = hat * wd + b.double()
    e_hat = (e_mean[:, None] + 2 * U * mid.abs()) * r[:, None] + mid.abs() * e_rstd[:, None]
    _check(y, want, _store(want, dtype) + e_hat * wd.abs() + 4 * U * (want.abs() + (hat * wd).abs() + b.double().abs()),
           "y")
    del want, e_hat, mid, hat
    # backward from the computed mean and rstd, taken as they are
    hat = (xd - mean.double()[:, None]) * rstd.double()[:, None]
    del xd
    rs = rstd.double()[:, None]
    dx, dw, db = bcl.layer_norm_bwd(x, w, mean, rstd, dy)
    gy = dy.double()
    gw = gy * wd
    along = (gw * hat).mean(-1, keepdim=True)
    want = rs * (gw - gw.mean(-1, keepdim=True) - hat * along)
    inner = gw.abs() + gw.abs().mean(-1, keepdim=True) + hat.abs() * (gw * hat).abs().mean(-1, keepdim=True)
    _check(dx, want, _store(want, dtype) + rs * (sum_err(d) + 16 * U) * inner, "dx")
    del want, inner, gw
    _check(dw, (gy * hat).sum(0), (rows + 22) * U * (gy * hat).abs().sum(0), "dw")
    _check(db, gy.sum(0), (rows + 16) * U * gy.abs().sum(0), "db")
    del gy, hat
    # over their own inputs, and again
    z = dy.clone()
    again = bcl.layer_norm_bwd(x, w, mean, rstd, z, dx=z)
    assert torch.equal(z, dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)
    bcl.layer_norm_fwd(x, w, b, EPS, y=x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,d", ROUNDS)
def test_layer_norm_over_several_rounds(rows, d, dtype):
    _run(rows, d, dtype)


@pytest.mark.parametrize("rows,d,dtype", LARGE)
def test_layer_norm_past_the_caches(rows, d, dtype):
    assert 2 * rows * d * {"f32": 4, "bf16": 2, "f16": 2}[dtype] > 320 << 20
    _run(rows, d, dtype)


def test_strided_rows_over_several_rounds():
    # rows of a wider buffer at an odd offset, each workgroup taking many
    g = torch.Generator(device=DEV).manual_seed(3)
    wide = torch.randn(5003, 1040, generator=g, device=DEV).to(torch.bfloat16)
    x = wide[:, 5:5 + 1027]
    w = torch.randn(1027, generator=g, device=DEV)
    y, m, r = bcl.layer_norm_fwd(x, w)
    y0, m0, r0 = bcl.layer_norm_fwd(x.contiguous(), w)
    assert torch.equal(y, y0) and torch.equal(m, m0) and torch.equal(r, r0)
    for a, b in zip(bcl.layer_norm_bwd(x, w, m, r, x), bcl.layer_norm_bwd(x.contiguous(), w, m, r, x.contiguous())):
        assert torch.equal(a, b)
