"""Operators of a fine-tuning step around the circulant layers.

Layer normalisation, token log-probabilities, the pairwise preference loss and
the clipped policy loss on vocabulary logits, and the global gradient norm with
clipping, on the HIP library ``lib/libfinetune.so`` (C ABI in
``include/finetune.h``, which holds the formulas).

Three layers, as for the circulant operators: calls that marshal arguments for
one entry point each (``layer_norm_fwd`` ...), autograd functions on them
(:func:`layer_norm`, :func:`token_logp`, :func:`preference_loss`,
:func:`policy_loss`), and the module :class:`LayerNorm` with
:func:`clip_grad_norm_` for a list of parameters.

Calls only enqueue work on the current stream of the tensors' device, or on
``stream``, where their temporary workspace is then allocated too.  There is
no CPU path.  Weights and statistics are float32; activations and logits may be
float32, bfloat16 or float16.
"""

from __future__ import annotations

import array
import ctypes
import functools
import os
from typing import NamedTuple

import torch

from .binding import RdfftError, _dtype_code

__all__ = [
    "FinetuneError",
    "finetune_lib",
    "finetune_lib_path",
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
_LIB = None

_I64 = ctypes.c_int64
_F64 = ctypes.c_double
_INT = ctypes.c_int
_VP = ctypes.c_void_p
_PI64 = ctypes.POINTER(_I64)


class _Logits(ctypes.Structure):
    _fields_ = [("data", _VP), ("labels", _VP), ("seqs", _I64), ("positions", _I64), ("vocab", _I64),
                ("seq_stride", _I64), ("pos_stride", _I64), ("dtype", _I64)]


class _DLogits(ctypes.Structure):
    _fields_ = [("data", _VP), ("seq_stride", _I64), ("pos_stride", _I64)]


class _Preference(ctypes.Structure):
    _fields_ = [("kind", _I64), ("average", _I64), ("beta", _F64), ("smoothing", _F64)]


class _Policy(ctypes.Structure):
    _fields_ = [("reduction", _I64), ("advantage_per_token", _I64), ("clip_low", _F64), ("clip_high", _F64),
                ("kl_coef", _F64)]


_PL, _PD, _PP, _PO = (ctypes.POINTER(t) for t in (_Logits, _DLogits, _Preference, _Policy))

# exported symbol -> (restype, argtypes); mirrors include/finetune.h
SIGNATURES = {
    "finetune_abi_version": (_INT, []),
    "finetune_status_string": (ctypes.c_char_p, [_INT]),
    "layer_norm_fwd": (_INT, [_VP] * 6 + [_I64] * 4 + [_F64, _INT, _VP]),
    "layer_norm_bwd_workspace": (_INT, [_I64, _I64, _PI64]),
    "layer_norm_bwd": (_INT, [_VP] * 9 + [_I64] * 6 + [_INT, _VP]),
    "finetune_logits_workspace": (_INT, [_PL, _PI64]),
    "token_logprob": (_INT, [_PL, _VP, _VP, _VP, _I64, _VP]),
    "token_logprob_bwd": (_INT, [_PL, _VP, _VP, _PD, _VP]),
    "preference_loss_fwd": (_INT, [_PL, _VP, _PP] + [_VP] * 6 + [_I64, _VP]),
    "preference_loss_bwd": (_INT, [_PL, _VP, _VP, _VP, _PD, _VP]),
    "preference_loss_step": (_INT, [_PL, _VP, _PP, _F64] + [_VP] * 5 + [_PD, _VP, _I64, _VP]),
    "policy_loss_fwd": (_INT, [_PL, _VP, _VP, _VP, _PO] + [_VP] * 5 + [_I64, _VP]),
    "policy_loss_bwd": (_INT, [_PL, _VP, _VP, _VP, _PD, _VP]),
    "policy_loss_step": (_INT, [_PL, _VP, _VP, _VP, _PO, _F64] + [_VP] * 4 + [_PD, _VP, _I64, _VP]),
    "grad_norm_workspace": (_INT, [_VP, _I64, _PI64]),
    "grad_norm": (_INT, [_VP, _I64, _VP, _VP, _I64, _VP]),
    "clip_grad_norm": (_INT, [_VP, _I64, _F64, _F64, _VP, _VP, _I64, _VP]),
}


def finetune_lib_path() -> str:
    return os.environ.get("FINETUNE_LIB", os.path.join(_HERE, "lib", "libfinetune.so"))


def finetune_lib() -> ctypes.CDLL:
    """Load libfinetune.so once; raise if it has not been built."""
    global _LIB
    if _LIB is None:
        path = finetune_lib_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} not found: build it with `python -m block_circulant_layers_amd.build` "
                "(there is no fallback implementation)"
            )
        cdll = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(cdll, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = cdll
    return _LIB


class FinetuneError(RdfftError):
    """A nonzero status of libfinetune.so (``status``)."""

    def __init__(self, func: str, status: int):
        msg = finetune_lib().finetune_status_string(status).decode()
        RuntimeError.__init__(self, f"{func} failed: status {status} ({msg})")
        self.status = status


def _call(name: str, t: torch.Tensor, *args) -> None:
    """The entry point `name` on the current stream of t's device."""
    fn = getattr(finetune_lib(), name)
    dev = t.get_device()
    if torch.cuda.current_device() == dev:
        st = fn(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch.cuda.current_stream().cuda_stream)
    if st != 0:
        raise FinetuneError(name, st)


def _query(name: str, *args) -> int:
    out = _I64(0)
    st = getattr(finetune_lib(), name)(*args, ctypes.byref(out))
    if st != 0:
        raise FinetuneError(name, st)
    return out.value


def _workspace(t: torch.Tensor, nbytes: int, ws: torch.Tensor | None) -> torch.Tensor:
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=t.device)
    if ws.device != t.device or not ws.is_contiguous():
        raise ValueError("ws must be contiguous and on the tensors' device")
    return ws


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


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _f32(name: str, t: torch.Tensor, shape, like: torch.Tensor) -> torch.Tensor:
    """t checked as a contiguous float32 array of `shape` on like's device."""
    if t.dtype != torch.float32 or t.shape != shape:
        raise ValueError(f"{name} must be float32 of shape {tuple(shape)}")
    if t.device != like.device:
        raise ValueError("tensors must be on one device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t


# ---------------------------------------------------------------------------
# layer normalisation
# ---------------------------------------------------------------------------
def _rows(name: str, t: torch.Tensor):
    """(rows, d, row stride) of a tensor whose last axis is contiguous and whose
    rows are evenly spaced."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU (there is no CPU path)")
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one axis")
    d = t.shape[-1]
    rows = t.numel() // d if d else 0
    if rows <= 1 or t.is_contiguous():
        if rows == 1 and d > 1 and t.stride(-1) != 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
        return rows, d, d
    if t.stride(-1) != 1 and d > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    want = None  # the stride that folds all leading axes into one
    step = 1
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if want is None:
            want = stride
        if stride != want * step:
            raise ValueError(f"the rows of {name} must be evenly spaced")
        step *= size
    return rows, d, want


def _same_rows(name: str, t: torch.Tensor, like: torch.Tensor) -> int:
    if t.dtype != like.dtype or t.shape != like.shape or t.device != like.device:
        raise ValueError(f"{name} must have the dtype, shape and device of x")
    return _rows(name, t)[2]


@_streamed
def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                   eps: float = 1e-5, y: torch.Tensor | None = None):
    """Returns (y, mean, rstd): the rows of x (last axis) normalised, scaled by
    ``weight`` and shifted by ``bias`` (float32 of the row's length, or None);
    mean and rstd (float32, one a row) are what the backward needs.  ``y`` may
    be x itself."""
    rows, d, xs = _rows("x", x)
    if weight is not None:
        _f32("weight", weight, (d,), x)
    if bias is not None:
        _f32("bias", bias, (d,), x)
    if y is None:
        y, ys = torch.empty(x.shape, dtype=x.dtype, device=x.device), d
    else:
        ys = _same_rows("y", y, x)
    stats = torch.empty((2,) + x.shape[:-1], dtype=torch.float32, device=x.device)
    mean, rstd = stats[0], stats[1]
    _call("layer_norm_fwd", x, x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), mean.data_ptr(),
          rstd.data_ptr(), rows, d, xs, ys, eps, _dtype_code(x))
    return y, mean, rstd


@_streamed
def layer_norm_bwd(x: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor, rstd: torch.Tensor,
                   dy: torch.Tensor, dx: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                   db: torch.Tensor | None = None, need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
                   ws: torch.Tensor | None = None):
    """Returns (dx, dw, db) for an upstream gradient dy (None for what is not
    needed).  dw and db (float32) are overwritten; ``dx`` may be dy itself."""
    rows, d, xs = _rows("x", x)
    dys = _same_rows("dy", dy, x)
    if weight is not None:
        _f32("weight", weight, (d,), x)
    _f32("mean", mean, x.shape[:-1], x)
    _f32("rstd", rstd, x.shape[:-1], x)
    dxs = d
    if not need_dx:
        dx = None
    elif dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        dxs = _same_rows("dx", dx, x)
    sums = []
    for name, t, need in (("dw", dw, need_dw), ("db", db, need_db)):
        if not need:
            sums.append(None)
        elif t is None:
            sums.append(torch.empty(d, dtype=torch.float32, device=x.device))
        else:
            sums.append(_f32(name, t, (d,), x))
    dw, db = sums
    nbytes = 0
    if dw is not None or db is not None:
        nbytes = _query("layer_norm_bwd_workspace", rows, d)
        ws = _workspace(x, nbytes, ws)
        nbytes = ws.numel() * ws.element_size()
    _call("layer_norm_bwd", x, x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(), dy.data_ptr(), _ptr(dx),
          _ptr(dw), _ptr(db), _ptr(ws), nbytes, rows, d, xs, dys, dxs, _dtype_code(x))
    return dx, dw, db


def _row_layout(t: torch.Tensor) -> torch.Tensor:
    """t itself where the kernels can address its rows, else a contiguous copy."""
    try:
        _, d, stride = _rows("x", t)
        return t if stride >= d else t.contiguous()
    except ValueError:
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
def _logits(logits: torch.Tensor, labels: torch.Tensor) -> _Logits:
    if not logits.is_cuda or not labels.is_cuda:
        raise ValueError("tensors must be on a GPU (there is no CPU path)")
    if logits.dim() != 3:
        raise ValueError("logits must have shape (sequences, positions, vocabulary)")
    seqs, positions, vocab = logits.shape
    if labels.dtype != torch.int64 or labels.shape != (seqs, positions):
        raise ValueError("labels must be int64 of shape (sequences, positions)")
    if labels.device != logits.device:
        raise ValueError("tensors must be on one device")
    if not labels.is_contiguous():
        raise ValueError("labels must be contiguous")
    ss, ps, last = logits.stride()
    if last != 1 and vocab > 1:
        raise ValueError("the vocabulary axis of logits must be contiguous")
    return _Logits(logits.data_ptr(), labels.data_ptr(), seqs, positions, vocab, ss, ps, _dtype_code(logits))


def _dlogits(logits: torch.Tensor, out: torch.Tensor | None):
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    elif out.shape != logits.shape or out.dtype != logits.dtype or out.device != logits.device:
        raise ValueError("dlogits must have the shape, dtype and device of logits")
    ss, ps, last = out.stride()
    if last != 1 and out.shape[2] > 1:
        raise ValueError("the vocabulary axis of dlogits must be contiguous")
    return out, _DLogits(out.data_ptr(), ss, ps)


def _logits_ws(logits: torch.Tensor, args: _Logits, ws: torch.Tensor | None):
    ws = _workspace(logits, _query("finetune_logits_workspace", ctypes.byref(args)), ws)
    return ws, ws.numel() * ws.element_size()


@_streamed
def token_logprob(logits: torch.Tensor, labels: torch.Tensor, ws: torch.Tensor | None = None):
    """Returns (logp, lse), float32 (sequences, positions): the log-probability
    of each label under the logits (sequences, positions, vocabulary), whose
    leading axes may be strided, and the log-sum-exp of the logits.  Both are 0
    where the label is IGNORE; those logits are not read."""
    args = _logits(logits, labels)
    out = torch.empty((2,) + labels.shape, dtype=torch.float32, device=logits.device)
    logp, lse = out[0], out[1]
    ws, n = _logits_ws(logits, args, ws)
    _call("token_logprob", logits, ctypes.byref(args), logp.data_ptr(), lse.data_ptr(), ws.data_ptr(), n)
    return logp, lse


@_streamed
def token_logprob_bwd(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, dlogp: torch.Tensor,
                      dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient for an upstream gradient of logp; ``dlogits`` may be
    the logits themselves, which are then replaced."""
    args = _logits(logits, labels)
    _f32("lse", lse, labels.shape, logits)
    _f32("dlogp", dlogp, labels.shape, logits)
    dlogits, dargs = _dlogits(logits, dlogits)
    _call("token_logprob_bwd", logits, ctypes.byref(args), lse.data_ptr(), dlogp.data_ptr(), ctypes.byref(dargs))
    return dlogits


class PreferenceLoss(NamedTuple):
    """loss (pairs), logratio (sequences), logp and lse (sequences, positions),
    slope (sequences): d loss / d logp of a sequence's unmasked positions."""

    loss: torch.Tensor
    logratio: torch.Tensor
    logp: torch.Tensor
    lse: torch.Tensor
    slope: torch.Tensor


_PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}


def _preference(logits, labels, ref_logp, beta, kind, label_smoothing, average):
    args = _logits(logits, labels)
    if logits.shape[0] % 2:
        raise ValueError("logits hold the chosen sequences and then as many rejected ones")
    if kind not in _PREFERENCE_KINDS:
        raise ValueError(f"kind must be one of {sorted(_PREFERENCE_KINDS)}")
    _f32("ref_logp", ref_logp, labels.shape, logits)
    n, t = labels.shape
    # one allocation for the small outputs: loss, logratio, slope, logp, lse
    buf = torch.empty(n // 2 + 2 * n + 2 * n * t, dtype=torch.float32, device=logits.device)
    loss, logratio, slope, logp, lse = buf.split((n // 2, n, n, n * t, n * t))
    out = PreferenceLoss(loss, logratio, logp.view(n, t), lse.view(n, t), slope)
    how = _Preference(_PREFERENCE_KINDS[kind], int(bool(average)), beta, label_smoothing)
    return args, how, out


@_streamed
def preference_loss_fwd(logits: torch.Tensor, labels: torch.Tensor, ref_logp: torch.Tensor, beta: float = 0.1,
                        kind: str = "sigmoid", label_smoothing: float = 0.0, average: bool = False,
                        ws: torch.Tensor | None = None) -> PreferenceLoss:
    """Pairwise preference loss of the chosen sequences (first half of the batch)
    against the rejected ones (second half), from token log-probabilities
    ``ref_logp`` of a reference model (float32 like labels).  ``kind``: "sigmoid"
    (with ``label_smoothing``), "hinge" or "ipo"; ``average``: log-ratios are
    means over a sequence's unmasked positions instead of sums."""
    args, how, r = _preference(logits, labels, ref_logp, beta, kind, label_smoothing, average)
    ws, n = _logits_ws(logits, args, ws)
    _call("preference_loss_fwd", logits, ctypes.byref(args), ref_logp.data_ptr(), ctypes.byref(how),
          r.loss.data_ptr(), r.logratio.data_ptr(), r.logp.data_ptr(), r.lse.data_ptr(), r.slope.data_ptr(),
          ws.data_ptr(), n)
    return r


@_streamed
def preference_loss_bwd(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, slope: torch.Tensor,
                        dloss: torch.Tensor, dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient for an upstream gradient dloss (pairs) from the
    forward's lse and slope; ``dlogits`` may be the logits themselves."""
    args = _logits(logits, labels)
    n = labels.shape[0]
    _f32("lse", lse, labels.shape, logits)
    _f32("slope", slope, (n,), logits)
    _f32("dloss", dloss, (n // 2,), logits)
    dlogits, dargs = _dlogits(logits, dlogits)
    _call("preference_loss_bwd", logits, ctypes.byref(args), lse.data_ptr(), slope.data_ptr(), dloss.data_ptr(),
          ctypes.byref(dargs))
    return dlogits


@_streamed
def preference_loss_step(logits: torch.Tensor, labels: torch.Tensor, ref_logp: torch.Tensor, beta: float = 0.1,
                         kind: str = "sigmoid", label_smoothing: float = 0.0, average: bool = False,
                         scale: float = 1.0, dlogits: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """:func:`preference_loss_fwd` and the logits' gradient of ``scale`` times
    the sum of the pairs' losses in one call; returns (PreferenceLoss, dlogits)."""
    args, how, r = _preference(logits, labels, ref_logp, beta, kind, label_smoothing, average)
    dlogits, dargs = _dlogits(logits, dlogits)
    ws, n = _logits_ws(logits, args, ws)
    _call("preference_loss_step", logits, ctypes.byref(args), ref_logp.data_ptr(), ctypes.byref(how), scale,
          r.loss.data_ptr(), r.logratio.data_ptr(), r.logp.data_ptr(), r.lse.data_ptr(), r.slope.data_ptr(),
          ctypes.byref(dargs), ws.data_ptr(), n)
    return r, dlogits


class PolicyLoss(NamedTuple):
    """loss and kl (scalars), logp, lse and slope (sequences, positions), slope
    being d loss / d logp."""

    loss: torch.Tensor
    kl: torch.Tensor
    logp: torch.Tensor
    lse: torch.Tensor
    slope: torch.Tensor


_POLICY_REDUCTIONS = {"token": 0, "sequence": 1, "sum": 2}


def _policy(logits, labels, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef, reduction):
    args = _logits(logits, labels)
    if reduction not in _POLICY_REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(_POLICY_REDUCTIONS)}")
    n, t = labels.shape
    _f32("old_logp", old_logp, labels.shape, logits)
    if ref_logp is not None:
        _f32("ref_logp", ref_logp, labels.shape, logits)
    per_token = advantages.shape == labels.shape and (t != 1 or advantages.dim() == 2)
    if not per_token and advantages.shape not in ((n,), (n, 1)):
        raise ValueError("advantages must have shape (sequences,), (sequences, 1) or (sequences, positions)")
    _f32("advantages", advantages, advantages.shape, logits)
    # one allocation for the small outputs: stats, logp, lse, slope
    buf = torch.empty(2 + 3 * n * t, dtype=torch.float32, device=logits.device)
    stats, logp, lse, slope = buf.split((2, n * t, n * t, n * t))
    out = PolicyLoss(stats[0], stats[1], logp.view(n, t), lse.view(n, t), slope.view(n, t))
    how = _Policy(_POLICY_REDUCTIONS[reduction], int(per_token), clip_low, clip_high, kl_coef)
    return args, how, out


@_streamed
def policy_loss_fwd(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                    ref_logp: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                    kl_coef: float = 0.0, reduction: str = "token", ws: torch.Tensor | None = None) -> PolicyLoss:
    """Clipped policy loss of sampled tokens ``labels`` with log-probabilities
    ``old_logp`` when they were sampled and ``advantages`` per sequence or
    token, plus ``kl_coef`` times the KL estimate against ``ref_logp``.
    ``reduction``: "token" (mean over unmasked positions), "sequence" (mean over
    sequences of their means) or "sum"."""
    args, how, r = _policy(logits, labels, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef, reduction)
    ws, n = _logits_ws(logits, args, ws)
    _call("policy_loss_fwd", logits, ctypes.byref(args), old_logp.data_ptr(), _ptr(ref_logp), advantages.data_ptr(),
          ctypes.byref(how), r.loss.data_ptr(), r.logp.data_ptr(), r.lse.data_ptr(), r.slope.data_ptr(),
          ws.data_ptr(), n)
    return r


@_streamed
def policy_loss_bwd(logits: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, slope: torch.Tensor,
                    dloss: torch.Tensor, dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient for an upstream gradient dloss (one float32) from
    the forward's lse and slope; ``dlogits`` may be the logits themselves."""
    args = _logits(logits, labels)
    _f32("lse", lse, labels.shape, logits)
    _f32("slope", slope, labels.shape, logits)
    if dloss.numel() != 1:
        raise ValueError("dloss must hold one value")
    _f32("dloss", dloss, dloss.shape, logits)
    dlogits, dargs = _dlogits(logits, dlogits)
    _call("policy_loss_bwd", logits, ctypes.byref(args), lse.data_ptr(), slope.data_ptr(), dloss.data_ptr(),
          ctypes.byref(dargs))
    return dlogits


@_streamed
def policy_loss_step(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                     ref_logp: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                     kl_coef: float = 0.0, reduction: str = "token", scale: float = 1.0,
                     dlogits: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """:func:`policy_loss_fwd` and the logits' gradient of ``scale`` times the
    loss in one call; returns (PolicyLoss, dlogits)."""
    args, how, r = _policy(logits, labels, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef, reduction)
    dlogits, dargs = _dlogits(logits, dlogits)
    ws, n = _logits_ws(logits, args, ws)
    _call("policy_loss_step", logits, ctypes.byref(args), old_logp.data_ptr(), _ptr(ref_logp), advantages.data_ptr(),
          ctypes.byref(how), scale, r.loss.data_ptr(), r.logp.data_ptr(), r.lse.data_ptr(), r.slope.data_ptr(),
          ctypes.byref(dargs), ws.data_ptr(), n)
    return r, dlogits


def _logits_layout(t: torch.Tensor) -> torch.Tensor:
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class _LogitLoss(torch.autograd.Function):
    """A loss on logits whose backward is one call from (lse, slope).  With
    ``inplace`` the gradient replaces the logits in their own buffer."""

    @staticmethod
    def forward(ctx, logits, labels, fwd, bwd, inplace):
        logits = _logits_layout(logits)
        outs, lse, slope = fwd(logits, labels)
        # a buffer that the backward itself overwrites is kept beside the saved tensors, good for one backward
        ctx.save_for_backward(labels, lse, slope, None if inplace else logits)
        ctx.logits, ctx.bwd = logits if inplace else None, bwd
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
        d = ctx.bwd(logits, labels, lse, slope, dloss.float().contiguous(), dlogits=target)
        return d, None, None, None, None


def token_logp(logits: torch.Tensor, labels: torch.Tensor, inplace: bool = False) -> torch.Tensor:
    """Differentiable token log-probabilities (sequences, positions) of labels;
    ``inplace``: the backward writes the gradient over the logits."""

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
    logits."""

    def fwd(x, y):
        r = preference_loss_fwd(x, y, ref_logp.contiguous(), beta, kind, label_smoothing, average)
        return (r.loss, r.logratio), r.lse, r.slope

    return _LogitLoss.apply(logits, labels.contiguous(), fwd, preference_loss_bwd, inplace)


def policy_loss(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
                ref_logp: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, reduction: str = "token", inplace: bool = False):
    """Differentiable clipped policy loss: returns (loss, kl); ``inplace``: the
    backward writes the gradient over the logits."""

    def fwd(x, y):
        r = policy_loss_fwd(x, y, old_logp.contiguous(), advantages.contiguous(),
                            None if ref_logp is None else ref_logp.contiguous(), clip_low, clip_high, kl_coef,
                            reduction)
        return (r.loss, r.kl), r.lse, r.slope

    return _LogitLoss.apply(logits, labels.contiguous(), fwd, policy_loss_bwd, inplace)


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------
def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one block of memory, in any order of axes."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != want:
            return False
        want *= size
    return True


_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _tensor_table(grads, out) -> array.array:
    """(grad, out, count, dtype) of every tensor as the C ABI's array."""
    table = []
    dev = grads[0].get_device()
    for g, o in zip(grads, out):
        code = _CODES.get(g.dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {g.dtype}: use float32, bfloat16 or float16")
        if g.get_device() != dev or dev < 0:
            raise ValueError("tensors must be on one GPU (there is no CPU path)")
        p = g.data_ptr()
        if not _dense(g):
            raise ValueError("gradients must fill one block of memory each")
        if o is g:
            q = p
        else:
            if o.dtype != g.dtype or o.get_device() != dev or o.shape != g.shape or o.stride() != g.stride():
                raise ValueError("out must match the gradients in dtype, device, shape and strides")
            q = o.data_ptr()
        table += (p, q, g.numel(), code)
    return array.array("q", table)


def _norm_call(name, grads, out, extra, norm, ws):
    grads = list(grads)
    out = grads if out is None else list(out)
    if not grads:
        raise ValueError("there are no gradient tensors")
    if len(out) != len(grads):
        raise ValueError("out must have one tensor per gradient")
    first = grads[0]
    table = _tensor_table(grads, out)
    ptr, n = table.buffer_info()[0], len(grads)
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=first.device)
    elif norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != first.device:
        raise ValueError("norm must hold one float32 on the gradients' device")
    ws = _workspace(first, _query("grad_norm_workspace", ptr, n), ws)
    _call(name, first, ptr, n, *extra, norm.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return norm


@_streamed
def grad_norm(grads, norm: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """The 2-norm of all gradient tensors together, a float32 on their device."""
    return _norm_call("grad_norm", grads, None, (), norm, ws)


@_streamed
def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6, out=None, norm: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None) -> torch.Tensor:
    """Scale the gradient tensors by min(1, max_norm / (norm + eps)), in place or
    into the tensors ``out``, and return their 2-norm (before clipping), a
    float32 on their device; nothing waits for the GPU."""
    return _norm_call("clip_grad_norm", grads, out, (max_norm, eps), norm, ws)


def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """:func:`clip_grad_norm` in place on the gradients that ``parameters``
    hold; a zero norm if none holds one."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    return clip_grad_norm(grads, max_norm, eps) if grads else torch.zeros(())
