"""GPU tests of what the fine-tuning operators overwrite: autograd is told, and
a value that the graph still needs raises instead of being read changed."""

from __future__ import annotations

import pytest
import torch

import block_circulant_layers_amd as bcl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(5)
    base = torch.randn(4, 5, 300, generator=g, device=DEV).to(dtype).requires_grad_(True)
    labels = torch.randint(0, 300, (4, 5), generator=g, device=DEV)
    ref = torch.randn(4, 5, generator=g, device=DEV) - 6.0
    return base, labels, ref, torch.randn(4, generator=g, device=DEV)


def _loss(kind, z, labels, ref, adv, **kw):
    if kind == "logp":
        return bcl.token_logp(z, labels, **kw).sum()
    if kind == "preference":
        return bcl.preference_loss(z, labels, ref, **kw)[0].sum()
    return bcl.policy_loss(z, labels, ref, adv, **kw)[0]


KINDS = ["logp", "preference", "policy"]


@pytest.mark.parametrize("kind", KINDS)
def test_two_losses_over_one_buffer(kind):
    base, labels, ref, adv = _case()
    z = base * 1.0
    total = _loss(kind, z, labels, ref, adv, inplace=True) + _loss("logp", z, labels, ref, adv, inplace=True)
    with pytest.raises(RuntimeError, match="modified"):
        total.backward()


@pytest.mark.parametrize("kind", KINDS)
def test_a_gradient_over_logits_that_others_saved(kind):
    base, labels, ref, adv = _case()
    z = base * 1.0
    other = z.square().sum()  # its backward runs after the loss's, which was made last
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (other + _loss(kind, z, labels, ref, adv, inplace=True)).backward()
    # a loss that does not overwrite them may stand beside any other
    base, labels, ref, adv = _case()
    z = base * 1.0
    (z.square().sum() + _loss(kind, z, labels, ref, adv)).backward()
    alone = base.detach().requires_grad_(True)
    _loss(kind, alone * 1.0, labels, ref, adv).backward()
    want = alone.grad.double() + 2 * base.detach().double()
    # two fp32 terms of magnitude 3 at most, each rounded, and their sum's rounding
    assert float((base.grad.double() - want).abs().max()) <= 1e-6 * float(want.abs().max())


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_logits_changed_before_the_backward(kind, inplace):
    base, labels, ref, adv = _case()
    z = base * 1.0
    loss = _loss(kind, z, labels, ref, adv, inplace=inplace)
    with torch.no_grad():
        z.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified"):
        loss.backward()


@pytest.mark.parametrize("kind", KINDS)
def test_inplace_gradient_is_the_other_ones(kind):
    # rows that the kernels cannot address go through a copy, which the gradient replaces instead
    for layout in (lambda t: t * 1.0, lambda t: (t * 1.0).transpose(1, 2).contiguous().transpose(1, 2)):
        grads = []
        for inplace in (False, True):
            base, labels, ref, adv = _case()
            _loss(kind, layout(base), labels, ref, adv, inplace=inplace).backward()
            grads.append(base.grad)
        assert torch.equal(*grads)


def test_calls_count_what_they_overwrite():
    base, labels, ref, adv = _case()
    x = base.detach().clone()
    w = torch.ones(300, device=DEV)

    def grows(call, *tensors):
        before = [t._version for t in tensors]
        call()
        assert [t._version - b for t, b in zip(tensors, before)] == [1] * len(tensors)

    y, mean, rstd = bcl.layer_norm_fwd(x, w)
    dy, dw, db = torch.randn_like(x), torch.empty_like(w), torch.empty_like(w)
    grows(lambda: bcl.layer_norm_fwd(x, w, y=y), y)
    grows(lambda: bcl.layer_norm_bwd(x, w, mean, rstd, dy, dx=dy, dw=dw, db=db), dy, dw, db)
    out = x.clone()
    grows(lambda: bcl.preference_loss_step(out, labels, ref, dlogits=out), out)
    grows(lambda: bcl.policy_loss_step(x, labels, ref, adv, dlogits=out), out)
    logp, lse = bcl.token_logprob(x, labels)
    grows(lambda: bcl.token_logprob_bwd(x, labels, lse, logp, dlogits=out), out)
    r = bcl.preference_loss_fwd(x, labels, ref)
    grows(lambda: bcl.preference_loss_bwd(x, labels, r.lse, r.slope, torch.ones(2, device=DEV), dlogits=out), out)
    p = bcl.policy_loss_fwd(x, labels, ref, adv)
    grows(lambda: bcl.policy_loss_bwd(x, labels, p.lse, p.slope, torch.ones((), device=DEV), dlogits=out), out)
    a, b, norm = torch.randn(100, device=DEV), torch.randn(7, device=DEV), torch.empty((), device=DEV)
    grows(lambda: bcl.clip_grad_norm([a, b], 0.1, norm=norm), a, b, norm)
    before = a._version
    grows(lambda: bcl.clip_grad_norm([a], 0.1, out=[out.view(-1)[:100]]), out)
    grows(lambda: bcl.grad_norm([a], norm=norm), norm)
    assert a._version == before and x._version == 0


def test_calls_in_inference_mode():
    base, labels, ref, adv = _case()
    with torch.inference_mode():
        x = base * 1.0
        w = torch.ones(300, device=DEV)
        y, mean, rstd = bcl.layer_norm_fwd(x, w)
        bcl.layer_norm_fwd(x, w, y=y)
        want = bcl.policy_loss(x, labels, ref, adv)[0]
        assert torch.equal(bcl.policy_loss(x, labels, ref, adv, inplace=True)[0], want)
        _, d = bcl.policy_loss_step(x, labels, ref, adv)
        bcl.policy_loss_step(x, labels, ref, adv, dlogits=x)
        assert torch.equal(x, d)
        bcl.clip_grad_norm([x], 1e-3)
    # a tensor made in inference mode may be overwritten outside it too, as before
    bcl.clip_grad_norm([x], 1e-4)
    assert abs(float(x.double().norm()) - 1e-4) <= 2e-7 or float(x.double().norm()) <= 1e-4
