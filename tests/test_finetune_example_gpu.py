"""The fine-tuning example end to end on the GPU: the losses fall, and its
gradients are those of the same model in plain float32 operations."""

from __future__ import annotations

import pytest
import torch

import block_circulant_layers_amd as bcl
from examples import finetune_adapters as ex

pytestmark = pytest.mark.gpu


def test_losses_fall():
    first, last, policy = ex.main(["--steps", "12", "--dim", "128", "--vocab", "1009"])
    assert last < 0.8 * first and policy[-1] < policy[0]


def test_gradients_against_plain_operations():
    dev = "cuda:0"
    model = ex.Model(257, 64, blocks=2, p=16, device=dev, dtype=torch.float32)
    with torch.no_grad():
        for a in model.adapters:
            a.c.normal_(0.0, 0.1, generator=torch.Generator(device=dev).manual_seed(3))
    tokens, labels = ex.batch(3, 12, 257, dev, seed=2)
    with torch.no_grad():
        ref, _ = bcl.token_logprob(model(tokens), labels)
        ref += 0.1 * torch.randn(ref.shape, generator=torch.Generator(device=dev).manual_seed(4), device=dev)
    loss, _ = bcl.preference_loss(model(tokens), labels, ref, beta=0.3)
    loss.mean().backward()
    got = [p.grad.double() for p in model.trained()]

    # the same model in float64: dense circulant products, torch's norm, softmax and autograd
    params = [p.detach().double().requires_grad_(True) for p in model.trained()]
    by_id = {id(p): q for p, q in zip(model.trained(), params)}

    def circulant(c, x):
        q, k, p = c.shape
        at = (torch.arange(p, device=dev)[:, None] - torch.arange(p, device=dev)[None, :]) % p
        w = c[:, :, at].permute(0, 2, 1, 3).reshape(q * p, k * p)
        return x @ w.t()

    h = model.embed.double()[tokens]
    for w, norm, adapter in zip(model.shared, model.norms, model.adapters):
        n = torch.nn.functional.layer_norm(h, (64,), by_id[id(norm.weight)], by_id[id(norm.bias)], norm.eps)
        h = h + torch.nn.functional.gelu(n @ w.double() + circulant(by_id[id(adapter.c)], n))
    norm = model.norms[-1]
    n = torch.nn.functional.layer_norm(h, (64,), by_id[id(norm.weight)], by_id[id(norm.bias)], norm.eps)
    logp = torch.log_softmax(n @ model.head.double().t(), -1).gather(2, labels.clamp(min=0)[..., None])[..., 0]
    gap = torch.where(labels != bcl.IGNORE, logp - ref.double(), 0.0).sum(-1)
    want = -torch.nn.functional.logsigmoid(0.3 * (gap[:3] - gap[3:]))
    assert torch.allclose(loss.double(), want, rtol=1e-4, atol=1e-5)
    want.mean().backward()
    for g, p in zip(got, params):
        # float32 through three blocks: about a hundred roundings of 6e-8 on the way, normwise
        assert float((g - p.grad).norm()) <= 1e-4 * float(p.grad.norm())
