"""Fine-tuning steps of block-circulant adapters on preference pairs and on sampled answers.

A small frozen language model (embedding, blocks of layer norm and a frozen
projection, a vocabulary head) gets a block-circulant adapter beside each
projection; only the adapters and the norms' weights train.  One step of each
kind runs everything the package has for it:

  * layer norm forward and backward (``LayerNorm``),
  * the circulant layer (``BlockCirculantLinear``),
  * the preference loss on chosen and rejected answers, or the clipped policy
    loss on answers with advantages, its gradient written over the logits,
  * the global gradient norm and clipping over all adapters,
  * a plain gradient step.

    python examples/finetune_adapters.py [--steps 20] [--dim 256] [--vocab 4001]

Synthetic tokens: chosen answers repeat a pattern, rejected ones are random, so
the printed losses fall and the margin between the two kinds rises.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_circulant_layers_amd as bcl  # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, vocab: int, dim: int, blocks: int, p: int, device, dtype=torch.bfloat16):
        super().__init__()
        g = torch.Generator(device=device).manual_seed(0)

        def frozen(*shape, scale):
            return torch.nn.Parameter(torch.randn(*shape, generator=g, device=device).mul_(scale).to(dtype),
                                      requires_grad=False)

        self.embed = frozen(vocab, dim, scale=1.0)
        self.head = frozen(vocab, dim, scale=dim**-0.5)
        self.shared = torch.nn.ParameterList([frozen(dim, dim, scale=dim**-0.5) for _ in range(blocks)])
        self.norms = torch.nn.ModuleList([bcl.LayerNorm(dim, device=device) for _ in range(blocks + 1)])
        self.adapters = torch.nn.ModuleList(
            [bcl.BlockCirculantLinear(dim, dim, p, device=device, generator=g) for _ in range(blocks)])
        with torch.no_grad():
            for a in self.adapters:
                a.c.zero_()  # the adapted model starts as the frozen one

    def forward(self, tokens: torch.Tensor) -> torch.Tensor:
        h = self.embed[tokens]
        for w, norm, adapter in zip(self.shared, self.norms, self.adapters):
            n = norm(h)
            h = h + torch.nn.functional.gelu(n @ w + adapter(n))
        return self.norms[-1](h) @ self.head.t()

    def trained(self):
        return [p for p in self.parameters() if p.requires_grad]


def batch(pairs: int, t: int, vocab: int, device, seed: int):
    """Tokens and labels of `pairs` chosen and `pairs` rejected sequences: a prompt
    (masked), an answer, padding (masked); labels are the next tokens."""
    g = torch.Generator(device=device).manual_seed(seed)
    tokens = torch.randint(0, vocab, (2 * pairs, t + 1), generator=g, device=device)
    start = t // 3
    for i in range(start, t + 1):  # a chosen answer follows a rule of the token before it
        tokens[:pairs, i] = (tokens[:pairs, i - 1] * 7 + 3) % 64
    labels = tokens[:, 1:].clone()
    labels[:, : start - 1] = bcl.IGNORE
    ends = torch.randint(t // 2, t + 1, (2 * pairs, 1), generator=g, device=device)
    labels[torch.arange(t, device=device) >= ends] = bcl.IGNORE
    return tokens[:, :-1].contiguous(), labels


def update(model: Model, lr: float, max_norm: float) -> torch.Tensor:
    params = model.trained()
    norm = bcl.clip_grad_norm_(params, max_norm)
    with torch.no_grad():
        for p in params:
            p.sub_(p.grad, alpha=lr)
            p.grad = None
    return norm


def preference_step(model: Model, tokens, labels, ref_logp, lr: float):
    loss, ratio = bcl.preference_loss(model(tokens), labels, ref_logp, beta=0.1, inplace=True)
    loss.mean().backward()
    norm = update(model, lr, 1.0)
    n = len(loss)
    return loss.detach().mean(), (ratio[:n] - ratio[n:]).mean(), norm


def policy_step(model: Model, tokens, labels, old_logp, ref_logp, advantages, lr: float):
    loss, kl = bcl.policy_loss(model(tokens), labels, old_logp, advantages, ref_logp=ref_logp, kl_coef=0.02,
                               inplace=True)
    loss.backward()
    return loss.detach(), kl, update(model, lr, 1.0)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=4001)
    ap.add_argument("--pairs", type=int, default=8)
    ap.add_argument("--positions", type=int, default=48)
    a = ap.parse_args(argv)
    device = "cuda:0"
    model = Model(a.vocab, a.dim, blocks=3, p=a.dim // 4, device=device)
    tokens, labels = batch(a.pairs, a.positions, a.vocab, device, seed=1)
    with torch.no_grad():
        ref_logp, _ = bcl.token_logprob(model(tokens), labels)
    first = last = None
    for i in range(a.steps):
        loss, margin, norm = preference_step(model, tokens, labels, ref_logp, lr=0.5)
        last = float(loss)
        first = last if first is None else first
        print(f"preference step {i}: loss {last:.4f} margin {float(margin):.3f} gradient norm {float(norm):.3f}")
    with torch.no_grad():
        old_logp, _ = bcl.token_logprob(model(tokens), labels)
    advantages = torch.cat([torch.ones(a.pairs, device=device), -torch.ones(a.pairs, device=device)])
    policy = []
    for i in range(a.steps):
        loss, kl, norm = policy_step(model, tokens, labels, old_logp, ref_logp, advantages, lr=0.5)
        policy.append(float(loss))
        print(f"policy step {i}: loss {policy[-1]:.4f} kl {float(kl):.4f} gradient norm {float(norm):.3f}")
    return first, last, policy


if __name__ == "__main__":
    main()
