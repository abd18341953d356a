"""Operators of a fine-tuning step around the circulant layers.

Layer normalisation, token log-probabilities, the pairwise preference loss and
the clipped policy loss on vocabulary logits, and the global gradient norm with
clipping, on the HIP library ``lib/libfinetune.so`` (C ABI in
``include/finetune.h``, which holds the formulas).

Three layers, as for the circulant operators: calls that stand for one entry
point each (``layer_norm_fwd`` ...; their arguments are checked and marshalled
by the module ``lib/_finetune_host.so``), autograd functions on them
(:func:`layer_norm`, :func:`token_logp`, :func:`preference_loss`,
:func:`policy_loss`), and the module :class:`LayerNorm` with
:func:`clip_grad_norm_` for a list of parameters.

Calls only enqueue work on the current stream of the tensors' device, or on
``stream``, where their temporary workspace is then allocated too.  There is
no CPU path.  A tensor of the caller's that a call overwrites counts as modified
in place, so that autograd refuses a backward that still needs its old values.
Weights and statistics are float32; activations and logits may be
float32, bfloat16 or float16.  ``ws`` is a workspace to use instead of a new
one, of at least the bytes that the C ABI's queries give.
"""

from __future__ import annotations

import functools
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple

import torch

from .binding import RdfftError

__all__ = [
    "FinetuneError",
    "IGNORE",
    "layer_norm_fwd",
    "layer_norm_bwd",
    "layer_norm",
    "LayerNorm",
    "token_logprob",
    "token_logprob_bwd",
    "token_logp",
    "PreferenceLoss",
    "preference_loss_fwd",
    "preference_loss_bwd",
    "preference_loss_step",
    "preference_loss",
    "PolicyLoss",
    "policy_loss_fwd",
    "policy_loss_bwd",
    "policy_loss_step",
    "policy_loss",
    "grad_norm",
    "clip_grad_norm",
    "clip_grad_norm_",
]

IGNORE = -100  # label of a position that takes no part in a loss

_HERE = os.path.dirname(os.path.abspath(__file__))
_HOST = None


def _host():
    """Load the module on libfinetune.so once; raise if it has not been built."""
    global _HOST
    if _HOST is None:
        path = os.path.join(_HERE, "lib", "_finetune_host.so")
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} not found: build it with `python -m block_circulant_layers_amd.build` "
                "(there is no fallback implementation)"
            )
        loader = importlib.machinery.ExtensionFileLoader("_finetune_host", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_finetune_host", path,
                                                                                        loader=loader))
        loader.exec_module(module)
        _HOST = module
    return _HOST


class FinetuneError(RdfftError):
    """A nonzero status of libfinetune.so (``status``)."""

    def __init__(self, func: str, status: int):
        RuntimeError.__init__(self, f"{func} failed: status {status} ({_host().status_string(status)})")
        self.status = status


def _streamed(fn):
    """`stream=...` runs the call with that stream current, so that what the
    call allocates belongs to the stream that uses it."""

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return fn(*args, **kw)

    return call


# ---------------------------------------------------------------------------
# layer normalisation
# ---------------------------------------------------------------------------
@_streamed
def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                   eps: float = 1e-5, y: torch.Tensor | None = None):
    """Returns (y, mean, rstd): the rows of x (last axis) normalised, scaled by
    ``weight`` and shifted by ``bias`` (float32 of the row's length, or None);
    mean and rstd (float32, one a row) are what the backward needs.  The last
    axis must be contiguous and the rows evenly spaced.  ``y`` may be x itself."""
    return _host().layer_norm_fwd(x, weight, bias, eps, y)


@_streamed
def layer_norm_bwd(x: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor, rstd: torch.Tensor,
                   dy: torch.Tensor, dx: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                   db: torch.Tensor | None = None, need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
                   ws: torch.Tensor | None = None):
    """Returns (dx, dw, db) for an upstream gradient dy (None for what is not
    needed).  dw and db (float32) are overwritten; ``dx`` may be dy itself."""
    return _host().layer_norm_bwd(x, weight, mean, rstd, dy, dx, dw, db, need_dx, need_dw, need_db, ws)


def _row_layout(t: torch.Tensor) -> torch.Tensor:
    """t itself where the kernels can address its rows, else a contiguous copy."""
    if t.is_contiguous():
        return t
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]:
        return t
    return t.contiguous()


class LayerNormFunction(torch.autograd.Function):
    """Layer normalisation; dx, dw and db from one backward call."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x = _row_layout(x)
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if not any(need[:3]):
            return None, None, None, None
        dx, dw, db = layer_norm_bwd(x, weight, mean, rstd, _row_layout(dy), need_dx=need[0],
                                    need_dw=need[1] and weight is not None, need_db=need[2])
        return dx, dw, db, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer normalisation over the last axis of x."""
    return LayerNormFunction.apply(x, weight, bias, eps)


class LayerNorm(torch.nn.Module):
    """Layer normalisation over rows of d elements with float32 weight and
    (optionally) bias; activations may be float32, bfloat16 or float16."""

    def __init__(self, d: int, eps: float = 1e-5, bias: bool = True, device=None):
        super().__init__()
        self.d, self.eps = d, eps
        self.weight = torch.nn.Parameter(torch.ones(d, dtype=torch.float32, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(d, dtype=torch.float32, device=device)) if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return layer_norm(x, self.weight, self.bias, self.eps)


# ---------------------------------------------------------------------------
# losses on logits
# ---------------------------------------------------------------------------
@_streamed
def token_logprob(logits: torch.Tensor, labels: torch.Tensor, ws: torch.Tensor | None = None):
    """Returns (logp, lse), float32 (sequences, positions): the log-probability
    of each label under the logits (sequences, positions, vocabulary), whose
    leading axes may be strided, and the log-sum-exp of the logits.  Both are 0
    where the label is IGNORE; those logits are not read."""
    return _host().token_logprob(logits, labels, ws)


@_streamed
def token_logprob_bwd(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, dlogp: torch.Tensor,
                      dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient for an upstream gradient of logp; ``dlogits`` may be
    the logits themselves, which are then replaced."""
    return _host().token_logprob_bwd(logits, labels, lse, dlogp, dlogits)


class PreferenceLoss(NamedTuple):
    """loss (pairs), logratio (sequences), logp and lse (sequences, positions),
    slope (sequences): d loss / d logp of a sequence's unmasked positions."""

    loss: torch.Tensor
    logratio: torch.Tensor
    logp: torch.Tensor
    lse: torch.Tensor
    slope: torch.Tensor


_PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}


def _choice(name: str, value: str, table: dict) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}")
    return table[value]


@_streamed
def preference_loss_fwd(logits: torch.Tensor, labels: torch.Tensor, ref_logp: torch.Tensor, beta: float = 0.1,
                        kind: str = "sigmoid", label_smoothing: float = 0.0, average: bool = False,
                        ws: torch.Tensor | None = None) -> PreferenceLoss:
    """Pairwise preference loss of the chosen sequences (first half of the batch)
    against the rejected ones (second half), from token log-probabilities
    ``ref_logp`` of a reference model (float32 like labels).  ``kind``: "sigmoid"
    (with ``label_smoothing``), "hinge" or "ipo"; ``average``: log-ratios are
    means over a sequence's unmasked positions instead of sums."""
    kind = _choice("kind", kind, _PREFERENCE_KINDS)
    return PreferenceLoss(*_host().preference_loss(logits, labels, ref_logp, beta, kind, label_smoothing, average,
                                                   None, None, ws)[:5])


@_streamed
def preference_loss_bwd(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, slope: torch.Tensor,
                        dloss: torch.Tensor, dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient for an upstream gradient dloss (pairs) from the
    forward's lse and slope; ``dlogits`` may be the logits themselves."""
    return _host().preference_loss_bwd(logits, labels, lse, slope, dloss, dlogits)


@_streamed
def preference_loss_step(logits: torch.Tensor, labels: torch.Tensor, ref_logp: torch.Tensor, beta: float = 0.1,
                         kind: str = "sigmoid", label_smoothing: float = 0.0, average: bool = False,
                         scale: float = 1.0, dlogits: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """:func:`preference_loss_fwd` and the logits' gradient of ``scale`` times
    the sum of the pairs' losses in one call; returns (PreferenceLoss, dlogits)."""
    kind = _choice("kind", kind, _PREFERENCE_KINDS)
    *r, d = _host().preference_loss(logits, labels, ref_logp, beta, kind, label_smoothing, average, scale, dlogits, ws)
    return PreferenceLoss(*r), d


class PolicyLoss(NamedTuple):
    """loss and kl (scalars), logp, lse and slope (sequences, positions), slope
    being d loss / d logp."""

    loss: torch.Tensor
    kl: torch.Tensor
    logp: torch.Tensor
    lse: torch.Tensor
    slope: torch.Tensor


_POLICY_REDUCTIONS = {"token": 0, "sequence": 1, "sum": 2}


@_streamed
def policy_loss_fwd(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                    ref_logp: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                    kl_coef: float = 0.0, reduction: str = "token", ws: torch.Tensor | None = None) -> PolicyLoss:
    """Clipped policy loss of sampled tokens ``labels`` with log-probabilities
    ``old_logp`` when they were sampled and ``advantages`` per sequence or
    token, plus ``kl_coef`` times the KL estimate against ``ref_logp``.
    ``reduction``: "token" (mean over unmasked positions), "sequence" (mean over
    sequences of their means) or "sum"."""
    reduction = _choice("reduction", reduction, _POLICY_REDUCTIONS)
    return PolicyLoss(*_host().policy_loss(logits, labels, old_logp, advantages, ref_logp, clip_low, clip_high,
                                           kl_coef, reduction, None, None, ws)[:5])


@_streamed
def policy_loss_bwd(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, slope: torch.Tensor,
                    dloss: torch.Tensor, dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient for an upstream gradient dloss (one float32) from
    the forward's lse and slope; ``dlogits`` may be the logits themselves."""
    return _host().policy_loss_bwd(logits, labels, lse, slope, dloss, dlogits)


@_streamed
def policy_loss_step(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                     ref_logp: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                     kl_coef: float = 0.0, reduction: str = "token", scale: float = 1.0,
                     dlogits: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """:func:`policy_loss_fwd` and the logits' gradient of ``scale`` times the
    loss in one call; returns (PolicyLoss, dlogits)."""
    reduction = _choice("reduction", reduction, _POLICY_REDUCTIONS)
    *r, d = _host().policy_loss(logits, labels, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef,
                                reduction, scale, dlogits, ws)
    return PolicyLoss(*r), d


def _logits_layout(t: torch.Tensor) -> torch.Tensor:
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class _LogitLoss(torch.autograd.Function):
    """A loss on logits whose backward is one call from (lse, slope).  With
    ``inplace`` the gradient replaces the logits in their own buffer."""

    @staticmethod
    def forward(ctx, logits, labels, fwd, bwd, inplace):
        logits = _logits_layout(logits)
        outs, lse, slope = fwd(logits, labels)
        # a buffer that the backward itself overwrites is kept beside the saved tensors, good for one backward, with
        # the version that autograd would otherwise check
        ctx.save_for_backward(labels, lse, slope, None if inplace else logits)
        ctx.logits, ctx.bwd = logits if inplace else None, bwd
        ctx.version = logits._version if inplace and not logits.is_inference() else None
        ctx.mark_non_differentiable(*outs[1:])
        return outs if len(outs) > 1 else outs[0]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, *_):
        labels, lse, slope, logits = ctx.saved_tensors
        target = None
        if logits is None:
            logits = target = ctx.logits
            ctx.logits = None
            if logits is None:
                raise RuntimeError("the loss was backpropagated before (its gradient replaced the logits)")
            if logits._version != ctx.version:
                raise RuntimeError("the logits were modified after the loss was computed from them (by another loss's "
                                   "inplace gradient, perhaps)")
        d = ctx.bwd(logits, labels, lse, slope, dloss.float().contiguous(), dlogits=target)
        return d, None, None, None, None


def token_logp(logits: torch.Tensor, labels: torch.Tensor, inplace: bool = False) -> torch.Tensor:
    """Differentiable token log-probabilities (sequences, positions) of labels;
    ``inplace``: the backward writes the gradient over the logits.  What else in
    the graph needs them, or another part of the tensor they are a view of,
    raises if its backward comes later."""

    def fwd(x, y):
        logp, lse = token_logprob(x, y)
        return (logp,), lse, lse

    def bwd(x, y, lse, _, dlogp, dlogits):
        return token_logprob_bwd(x, y, lse, dlogp, dlogits=dlogits)

    return _LogitLoss.apply(logits, labels.contiguous(), fwd, bwd, inplace)


def preference_loss(logits: torch.Tensor, labels: torch.Tensor, ref_logp: torch.Tensor, beta: float = 0.1,
                    kind: str = "sigmoid", label_smoothing: float = 0.0, average: bool = False,
                    inplace: bool = False):
    """Differentiable preference loss: returns (loss of each pair, log-ratio of
    each sequence); ``inplace``: the backward writes the gradient over the
    logits, as for :func:`token_logp`."""

    def fwd(x, y):
        r = preference_loss_fwd(x, y, ref_logp.contiguous(), beta, kind, label_smoothing, average)
        return (r.loss, r.logratio), r.lse, r.slope

    return _LogitLoss.apply(logits, labels.contiguous(), fwd, preference_loss_bwd, inplace)


def policy_loss(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                ref_logp: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, reduction: str = "token", inplace: bool = False):
    """Differentiable clipped policy loss: returns (loss, kl); ``inplace``: the
    backward writes the gradient over the logits, as for :func:`token_logp`."""

    def fwd(x, y):
        r = policy_loss_fwd(x, y, old_logp.contiguous(), advantages.contiguous(),
                            None if ref_logp is None else ref_logp.contiguous(), clip_low, clip_high, kl_coef,
                            reduction)
        return (r.loss, r.kl), r.lse, r.slope

    return _LogitLoss.apply(logits, labels.contiguous(), fwd, policy_loss_bwd, inplace)


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------
@_streamed
def grad_norm(grads, norm: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """The 2-norm of all gradient tensors together, a float32 on their device."""
    return _host().clip_grad_norm(grads if isinstance(grads, list) else list(grads), None, 0.0, None, norm, ws)


@_streamed
def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6, out=None, norm: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None) -> torch.Tensor:
    """Scale the gradient tensors by min(1, max_norm / (norm + eps)), in place or
    into the tensors ``out``, and return their 2-norm (before clipping), a
    float32 on their device; nothing waits for the GPU."""
    return _host().clip_grad_norm(grads if isinstance(grads, list) else list(grads), max_norm, eps,
                                  out if out is None or isinstance(out, list) else list(out), norm, ws)


def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """:func:`clip_grad_norm` in place on the gradients that ``parameters``
    hold; a zero norm if none holds one."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    return clip_grad_norm(grads, max_norm, eps) if grads else torch.zeros(())
