"""Operators of a transformer sublayer around the circulant layers.

Attention whose backward recomputes the probabilities, a learned relative
position bias by buckets (inside the attention, or as a tensor), and dropout
from a counter-based generator, on the HIP library ``lib/libfinetune.so`` (C ABI
in ``include/attention.h``, which holds the formulas).  Nothing of the size of
the score matrix or of a mask is stored between forward and backward.

As for the operators of :mod:`block_circulant_layers_amd.finetune`: calls that
stand for one entry point each (``attention_fwd`` ...), autograd functions on
them (:func:`attention`, :func:`relative_bias`, :func:`dropout`), and the
modules :class:`RelativeBias` and :class:`Dropout`.  Calls only enqueue work on
the current stream of the tensors' device, or on ``stream``; there is no CPU
path; a tensor of the caller's that a call overwrites counts as modified in
place; ``ws`` is a workspace to use instead of a new one.
"""

from __future__ import annotations

import torch

from .finetune import _host, _row_layout, _streamed

__all__ = [
    "attention_fwd",
    "attention_bwd",
    "attention",
    "relative_bias_fwd",
    "relative_bias_bwd",
    "relative_bias",
    "RelativeBias",
    "dropout_fwd",
    "dropout_bwd",
    "dropout",
    "Dropout",
]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
@_streamed
def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None, causal: bool = False,
                  key_begin: torch.Tensor | None = None, key_end: torch.Tensor | None = None,
                  bias: torch.Tensor | None = None, max_distance: int = 128, bidirectional: bool = True,
                  o: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Returns (o, lse) of q (batch, queries, heads, d) against k and v (batch,
    keys, key heads, d): o like q, and the log-sum-exp of each query's scores,
    float32 (batch, heads, queries).  d is at most 128; the last axis must be
    contiguous, the others may be strided.  Heads are a multiple of key heads and
    share them group by group.  ``scale``: 1 / sqrt(d) unless given.  ``causal``:
    query i sees keys up to i + keys - queries.  ``key_begin``, ``key_end``
    (int32, one a sequence): the keys that count; the others are not read.
    ``bias``: a float32 table (buckets, heads) of a relative position bias, with
    ``max_distance`` and ``bidirectional`` as for :func:`relative_bias`.  A query
    that sees no key gets zeros and an lse of -infinity."""
    return _host().attention_fwd(q, k, v, scale, causal, key_begin, key_end, bias, max_distance, bidirectional, o, ws)


@_streamed
def attention_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                  dout: torch.Tensor, scale: float | None = None, causal: bool = False,
                  key_begin: torch.Tensor | None = None, key_end: torch.Tensor | None = None,
                  bias: torch.Tensor | None = None, max_distance: int = 128, bidirectional: bool = True,
                  need_dbias: bool = True, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                  dv: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Returns (dq, dk, dv, dbias) for an upstream gradient dout of o, from the
    forward's o and lse; dk and dv sum over the heads that share a key head,
    dbias (float32 like the table) is None without a bias.  ``dq``, ``dk``,
    ``dv``: buffers to write, which may be parts of one fused buffer."""
    return _host().attention_bwd(q, k, v, o, lse, dout, scale, causal, key_begin, key_end, bias, max_distance,
                                 bidirectional, need_dbias, dq, dk, dv, ws)


def _last_contiguous(t: torch.Tensor) -> torch.Tensor:
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


class AttentionFunction(torch.autograd.Function):
    """Attention; dq, dk, dv and the bias table's gradient from one backward call."""

    @staticmethod
    def forward(ctx, q, k, v, bias, scale, causal, key_begin, key_end, max_distance, bidirectional):
        q, k, v = (_last_contiguous(t) for t in (q, k, v))
        table = None if bias is None else bias.contiguous()
        o, lse = attention_fwd(q, k, v, scale, causal, key_begin, key_end, table, max_distance, bidirectional)
        ctx.save_for_backward(q, k, v, o, lse, table, key_begin, key_end)
        ctx.how = scale, causal, max_distance, bidirectional
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse, table, key_begin, key_end = ctx.saved_tensors
        scale, causal, max_distance, bidirectional = ctx.how
        dq, dk, dv, dbias = attention_bwd(q, k, v, o, lse, _last_contiguous(dout), scale, causal, key_begin, key_end,
                                          table, max_distance, bidirectional, need_dbias=ctx.needs_input_grad[3])
        return dq, dk, dv, dbias, None, None, None, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None, causal: bool = False,
              key_begin: torch.Tensor | None = None, key_end: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, max_distance: int = 128, bidirectional: bool = True) -> torch.Tensor:
    """Differentiable attention, arguments as for :func:`attention_fwd`; keeps q,
    k, v, o and one float32 a query for the backward, no probabilities."""
    return AttentionFunction.apply(q, k, v, bias, scale, causal, key_begin, key_end, max_distance, bidirectional)


# ---------------------------------------------------------------------------
# relative position bias
# ---------------------------------------------------------------------------
@_streamed
def relative_bias_fwd(table: torch.Tensor, queries: int, keys: int, max_distance: int = 128,
                      bidirectional: bool = True, dtype: torch.dtype = torch.float32,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """The bias (heads, queries, keys) in ``dtype`` from a float32 table
    (buckets, heads): position key - query (the last query stands at the last
    key) picks the bucket.  Near positions have one each, others grow with the
    logarithm up to ``max_distance``; ``bidirectional``: half of the buckets for
    keys after the query, else those count as distance 0."""
    return _host().relative_bias_fwd(table, queries, keys, max_distance, bidirectional, dtype, out)


@_streamed
def relative_bias_bwd(dbias: torch.Tensor, buckets: int, max_distance: int = 128, bidirectional: bool = True,
                      dtable: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """The table's gradient, float32 (buckets, heads), from dbias ([batch,] heads,
    queries, keys), summed over the batch; leading axes may be strided."""
    return _host().relative_bias_bwd(dbias, buckets, max_distance, bidirectional, dtable, ws)


class RelativeBiasFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, queries, keys, max_distance, bidirectional, dtype):
        ctx.how = table.shape[0], max_distance, bidirectional
        return relative_bias_fwd(table.contiguous(), queries, keys, max_distance, bidirectional, dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dbias):
        return relative_bias_bwd(_last_contiguous(dbias), *ctx.how), None, None, None, None, None


def relative_bias(table: torch.Tensor, queries: int, keys: int, max_distance: int = 128, bidirectional: bool = True,
                  dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Differentiable :func:`relative_bias_fwd`."""
    return RelativeBiasFunction.apply(table, queries, keys, max_distance, bidirectional, dtype)


class RelativeBias(torch.nn.Module):
    """A learned relative position bias: a float32 table ``weight`` (buckets,
    heads).  Called with lengths it gives the bias as a tensor; ``attend`` is
    :func:`attention` with the table fused in."""

    def __init__(self, heads: int, buckets: int = 32, max_distance: int = 128, bidirectional: bool = True,
                 device=None):
        super().__init__()
        self.max_distance, self.bidirectional = max_distance, bidirectional
        self.weight = torch.nn.Parameter(torch.zeros(buckets, heads, dtype=torch.float32, device=device))

    def forward(self, queries: int, keys: int, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        return relative_bias(self.weight, queries, keys, self.max_distance, self.bidirectional, dtype)

    def attend(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, **kw) -> torch.Tensor:
        return attention(q, k, v, bias=self.weight, max_distance=self.max_distance,
                         bidirectional=self.bidirectional, **kw)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
def _seed_parts(seed):
    """(number, device tensor) of a seed that may be either."""
    return (0, seed) if isinstance(seed, torch.Tensor) else (seed, None)


@_streamed
def dropout_fwd(x: torch.Tensor, p: float, seed, offset: int = 0, residual: torch.Tensor | None = None,
                y: torch.Tensor | None = None) -> torch.Tensor:
    """Elements of x dropped with probability p (to 1 / 65536), the others scaled
    so that the mean stays, plus ``residual``.  The mask is a function of the
    element's index, ``seed`` and ``offset`` (0 .. 2^64 - 1; another offset is
    another mask) and stored nowhere.  A seed may be an int64 tensor of one
    element on the device, read when the kernel runs, so that replays of a graph
    can draw new masks.  Rows (last axis contiguous) must be evenly spaced;
    ``y`` may be x or the residual itself."""
    number, device = _seed_parts(seed)
    return _host().dropout(x, p, number, offset, device, residual, y, False)


@_streamed
def dropout_bwd(dy: torch.Tensor, p: float, seed, offset: int = 0, dx: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of x for an upstream gradient dy, with the forward's mask; ``dx`` may be dy itself."""
    number, device = _seed_parts(seed)
    return _host().dropout(dy, p, number, offset, device, None, dx, True)


class DropoutFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        ctx.p, ctx.offset = p, offset
        ctx.seed = None if isinstance(seed, torch.Tensor) else seed
        ctx.save_for_backward(None if ctx.seed is not None else seed)
        return dropout_fwd(_row_layout(x), p, seed, offset, None if residual is None else _row_layout(residual))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        (seed,) = ctx.saved_tensors
        dx = None
        if ctx.needs_input_grad[0]:
            dx = dropout_bwd(_row_layout(dy), ctx.p, seed if ctx.seed is None else ctx.seed, ctx.offset)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


def dropout(x: torch.Tensor, p: float, seed=None, offset: int = 0,
            residual: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable :func:`dropout_fwd`.  Without a ``seed`` one is drawn from
    torch's default CPU generator; a graph that is being captured would replay
    that one mask, so there a seed is required (a device tensor draws anew)."""
    if seed is None:
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("dropout in a captured graph needs a seed: a device tensor, or a number for one mask")
        seed = int(torch.empty((), dtype=torch.int64).random_())
    return DropoutFunction.apply(x, residual, p, seed, offset)


class Dropout(torch.nn.Module):
    """Dropout with an optional residual sum; without one the identity in
    evaluation.  ``seed`` and ``offset`` as for :func:`dropout`."""

    def __init__(self, p: float = 0.1):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be between 0 and 1")
        self.p = p

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, seed=None,
                offset: int = 0) -> torch.Tensor:
        if not self.training or self.p == 0.0:
            return x if residual is None else residual + x
        return dropout(x, self.p, seed, offset, residual)
