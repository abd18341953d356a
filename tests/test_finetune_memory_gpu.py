"""GPU tests of the memory behind what the fine-tuning calls return: a tensor
that is kept holds its own values and nothing of the call's workspace."""

from __future__ import annotations

import io

import pytest
import torch

import block_circulant_layers_amd as bcl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LEAST = 512  # bytes of the smallest block that torch's allocator hands out


def _calls(n, t, v):
    g = torch.Generator(device=DEV).manual_seed(6)
    z = torch.randn(n, t, v, generator=g, device=DEV)
    lab = torch.randint(0, v, (n, t), generator=g, device=DEV)
    ref, adv = torch.randn(n, t, generator=g, device=DEV), torch.randn(n, generator=g, device=DEV)
    return {
        "norm": lambda: bcl.layer_norm_fwd(z),
        "logprob": lambda: bcl.token_logprob(z, lab),
        "preference": lambda: bcl.preference_loss_fwd(z, lab, ref),
        "preference step": lambda: bcl.preference_loss_step(z, lab, ref)[0],
        "policy": lambda: bcl.policy_loss_fwd(z, lab, ref, adv),
        "policy step": lambda: bcl.policy_loss_step(z, lab, ref, adv)[0],
    }


@pytest.mark.parametrize("n,t,v", [(2, 3, 40), (2, 1, 9000), (4, 64, 300), (16, 700, 50), (2, 40, 9000)])
def test_results_hold_no_workspace(n, t, v):
    for name, call in _calls(n, t, v).items():
        for k, r in enumerate(call()):
            assert r.untyped_storage().nbytes() <= max(LEAST, r.numel() * r.element_size()), (name, k)


def test_kept_log_probabilities_cost_their_own_bytes():
    n, t, v = 64, 1024, 16
    call = _calls(n, t, v)["logprob"]
    call()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    kept = [call()[0] for _ in range(4)]
    assert torch.cuda.memory_allocated() - before <= 4 * (n * t * 4 + LEAST)
    buf = io.BytesIO()
    torch.save(kept[0], buf)
    assert buf.tell() <= n * t * 4 + 4096
