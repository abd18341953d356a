"""The sublayer operators under autograd, and a run of them together as a transformer sublayer uses them."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import block_circulant_layers_amd as bcl
from tests.attention_util import DEV, ao, f64, rng, stored

pytestmark = pytest.mark.gpu


def leaf(r, *shape, dtype="f32", scale=1.0):
    t, ref = stored(scale * r.standard_normal(shape), dtype)
    return t.to(DEV).requires_grad_(True), ref


def near(got, want, tol):
    """Normwise."""
    got = f64(got)
    assert np.linalg.norm(got - want) <= tol * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("layout", ["plain", "heads_first", "last_axis_strided", "expanded_gradient"])
def test_attention_gradients(layout):
    r = rng(40)
    b, tq, tk, hq, hk, d = 2, 40, 50, 4, 2, 32
    q, qr = leaf(r, b, tq, hq, d)
    k, kr = leaf(r, b, tk, hk, d)
    v, vr = leaf(r, b, tk, hk, d)
    table, tr = leaf(r, 8, hq)
    up, ur = stored(r.standard_normal((b, tq, hq, d)), "f32")
    args = [q, k, v]
    if layout == "heads_first":
        args = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in args]
    if layout == "last_axis_strided":
        args = [x.transpose(2, 3).contiguous().transpose(2, 3) for x in args]
    o = bcl.attention(*args, bias=table, max_distance=20, bidirectional=True)
    if layout == "expanded_gradient":
        ur = np.ones_like(ur)
        o.sum().backward()
    else:
        o.backward(up.to(DEV))
    bias = ao.relative_bias(tr, tq, tk, 20, True)
    _, _, p = ao.attention(qr, kr, vr, d**-0.5, ao.visible(b, tq, tk), bias)
    dq, dk, dv, ds = ao.attention_bwd(qr, kr, vr, p, ur, d**-0.5)
    scale = np.linalg.norm(ds)
    # fp32 throughout: sums of at most 100 terms of either sign
    for got, want in ((v.grad, dv), (q.grad, dq), (k.grad, dk), (table.grad, ao.relative_bias_bwd(ds, 8, 20, True))):
        assert np.linalg.norm(f64(got) - want) <= 2e-5 * np.linalg.norm(want) + 2e-5 * scale


def test_gradients_where_they_are_asked_for():
    r = rng(41)
    q, _ = leaf(r, 1, 20, 2, 16)
    k, _ = leaf(r, 1, 20, 2, 16)
    table, _ = leaf(r, 8, 2)
    o = bcl.attention(q, k.detach(), k.detach(), bias=table.detach(), max_distance=20)
    o.sum().backward()
    assert q.grad is not None and k.grad is None and table.grad is None
    with torch.no_grad():
        assert not bcl.attention(q, k, k).requires_grad
    bias = bcl.RelativeBias(2, buckets=8, max_distance=20, device=DEV)
    bias.attend(q, k, k).sum().backward()
    assert bias.weight.grad.shape == (8, 2)
    out = bias(20, 20, torch.bfloat16)
    assert out.dtype == torch.bfloat16 and out.shape == (2, 20, 20)
    bias.weight.grad = None
    out.float().mul(2.0).sum().backward()
    assert float(bias.weight.grad.sum()) == 2.0 * 2 * 400


def test_attention_refuses_changed_inputs():
    r = rng(42)
    q, _ = leaf(r, 1, 20, 2, 16)
    k = leaf(r, 1, 20, 2, 16)[0].detach()
    o = bcl.attention(q, k, k)
    bcl.dropout_fwd(k, 0.5, 1, y=k)  # overwritten by a call of the package
    with pytest.raises(RuntimeError, match="modified"):
        o.sum().backward()


def test_dropout_gradients():
    x, xr = leaf(rng(43), 30, 50)
    res, rr = leaf(rng(44), 30, 50)
    up, ur = stored(rng(45).standard_normal((30, 50)), "f32")
    y = bcl.dropout(x, 0.3, seed=5, offset=2, residual=res)
    near(y, ao.dropout(xr, 0.3, 5, 2, rr), 1e-6)
    y.backward(up.to(DEV))
    near(x.grad, ao.dropout(ur, 0.3, 5, 2), 1e-6)
    assert np.array_equal(f64(res.grad), ur)
    # drawn seeds follow torch's generator and differ from call to call
    torch.manual_seed(3)
    a, b = bcl.dropout(x, 0.5), bcl.dropout(x, 0.5)
    torch.manual_seed(3)
    assert torch.equal(a, bcl.dropout(x, 0.5)) and not torch.equal(a, b)
    module = bcl.Dropout(0.5)
    torch.manual_seed(3)
    assert torch.equal(a, module(x))
    # a seed tensor that changed between forward and backward is refused
    seed = torch.tensor([3], device=DEV)
    y = bcl.dropout(x, 0.5, seed=seed)
    seed += 1
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()


def test_dropout_in_a_capture_needs_a_seed():
    x = torch.ones(64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="seed"):
            bcl.dropout(x, 0.5)
        y = bcl.dropout(x, 0.5, seed=3)
    graph.replay()
    assert torch.equal(y, bcl.dropout_fwd(x, 0.5, 3))


def sublayer(x, norm, proj, out, bias, causal, ends, p, seed, heads):
    """x + dropout(projection(attention(projections(norm(x)))))"""
    b, t, dim = x.shape
    n = norm(x)
    q, k, v = (f(n.reshape(b * t, dim)).view(b, t, heads, dim // heads) for f in proj)
    o = bias.attend(q, k, v, causal=causal, key_end=ends)
    o = out(o.reshape(b * t, dim)).view(b, t, dim)
    return bcl.dropout(o, p, seed=seed, residual=x)


@pytest.mark.parametrize("causal", [False, True])
def test_sublayer_of_adapters(causal):
    """Norm, circulant projections, attention with its bias, dropout with the residual: forward and every gradient
    against float64 autograd of the same formulas."""
    torch.manual_seed(0)
    b, t, dim, heads, p = 3, 33, 64, 4, 16
    r = rng(46, causal)
    x, xr = leaf(r, b, t, dim)
    norm = bcl.LayerNorm(dim, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    proj = [bcl.BlockCirculantLinear(dim, dim, p, device=DEV, generator=g) for _ in range(3)]
    out = bcl.BlockCirculantLinear(dim, dim, p, device=DEV, generator=g)
    bias = bcl.RelativeBias(heads, buckets=8, max_distance=20, bidirectional=not causal, device=DEV)
    with torch.no_grad():
        bias.weight.normal_()
    ends = torch.tensor([t, 20, 0], device=DEV, dtype=torch.int32)
    y = sublayer(x, norm, proj, out, bias, causal, ends, 0.2, 9, heads)
    up, ur = stored(r.standard_normal((b, t, dim)), "f32")
    y.backward(up.to(DEV))

    leaves = {"x": torch.from_numpy(xr).requires_grad_(True), "w": torch.ones(dim, dtype=torch.float64, requires_grad=True),
              "b": torch.zeros(dim, dtype=torch.float64, requires_grad=True),
              "table": bias.weight.detach().cpu().double().requires_grad_(True)}
    cs = [m.c.detach().cpu().double().requires_grad_(True) for m in (*proj, out)]

    def circulant(n, c):
        spec = torch.fft.rfft(n.reshape(-1, dim // p, p)), torch.fft.rfft(c)
        return torch.fft.irfft(torch.einsum("bkf,qkf->bqf", *spec), n=p).reshape(-1, dim)

    n = torch.nn.functional.layer_norm(leaves["x"], (dim,), leaves["w"], leaves["b"], norm.eps)
    q, k, v = (circulant(n, c).view(b, t, heads, dim // heads).transpose(1, 2) for c in cs[:3])
    where = torch.from_numpy(ao.bucket_matrix(t, t, 8, 20, not causal))
    s = q @ k.transpose(2, 3) / (dim // heads) ** 0.5 + leaves["table"][where].permute(2, 0, 1)
    see = torch.from_numpy(ao.visible(b, t, t, causal, None, ends.cpu().numpy()))
    live = see.any(-1)
    s = torch.where(see | ~live[..., None], 0.0, -torch.inf)[:, None] + s
    o = (torch.softmax(s, -1) * live[:, None, :, None]) @ v
    o = circulant(o.transpose(1, 2).reshape(b * t, dim), cs[3]).view(b, t, dim)
    keep, scale = ao.dropout_keep(o.numel(), 0.2, 9, 0)
    want = leaves["x"] + o * torch.from_numpy(keep.reshape(b, t, dim)) * scale
    want.backward(torch.from_numpy(ur))
    # fp32 through six operators; each stays within a few 2^-24 of its terms' magnitudes
    near(y, want.detach().numpy(), 1e-5)
    grads = {"x": x.grad, "w": norm.weight.grad, "b": norm.bias.grad, "table": bias.weight.grad}
    for name, got in grads.items():
        near(got, leaves[name].grad.numpy(), 1e-4)
    for m, c in zip((*proj, out), cs):
        near(m.c.grad, c.grad.numpy(), 1e-4)
