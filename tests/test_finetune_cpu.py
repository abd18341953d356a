"""CPU checks of the fine-tuning operators: the C ABI's exports and argument
checks, the Python calls' refusals, the kernels on CPU threads under the
sanitizers, and the code object.

The pointers of the ABI cases are fake and never dereferenced: every call
carries an invalid argument or asks for no work, so no kernel is enqueued."""

from __future__ import annotations

import ctypes
import glob
import os
import re
import subprocess

import pytest
import torch

import block_circulant_layers_amd as bcl
from block_circulant_layers_amd import build
from tests.finetune_check import build_emu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "finetune.h")
I64, F64, INT, VP = ctypes.c_int64, ctypes.c_double, ctypes.c_int, ctypes.c_void_p

OK, NULL, SIZE, SHAPE, DTYPE, ALIGN, ALIAS = range(7)
F32, BF16, F16 = 0, 1, 2


class Logits(ctypes.Structure):
    _fields_ = [("data", VP), ("labels", VP), ("seqs", I64), ("positions", I64), ("vocab", I64),
                ("seq_stride", I64), ("pos_stride", I64), ("dtype", I64)]


class DLogits(ctypes.Structure):
    _fields_ = [("data", VP), ("seq_stride", I64), ("pos_stride", I64)]


class Preference(ctypes.Structure):
    _fields_ = [("kind", I64), ("average", I64), ("beta", F64), ("smoothing", F64)]


class Policy(ctypes.Structure):
    _fields_ = [("reduction", I64), ("per_token", I64), ("low", F64), ("high", F64), ("kl", F64)]


class Tensor(ctypes.Structure):
    _fields_ = [("grad", VP), ("out", VP), ("count", I64), ("dtype", I64)]


def _sources():
    csrc = os.path.join(ROOT, "block_circulant_layers_amd", "csrc", "finetune")
    return glob.glob(os.path.join(csrc, "*")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


@pytest.fixture(scope="module")
def L():
    newest = max(os.path.getmtime(s) for s in _sources())
    if any(not os.path.exists(p) or os.path.getmtime(p) < newest for p in (build.FINETUNE_LIB, build.FINETUNE_HOST)):
        build.build_finetune(verbose=False)
    lib = ctypes.CDLL(build.FINETUNE_LIB)
    lib.finetune_status_string.restype = ctypes.c_char_p
    return lib


def test_exports_every_declared_symbol(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(\w+)\s*\(", src, flags=re.M))
    assert names == {"finetune_abi_version", "finetune_status_string", "layer_norm_fwd", "layer_norm_bwd_workspace",
                     "layer_norm_bwd", "finetune_logits_workspace", "token_logprob", "token_logprob_bwd",
                     "preference_loss_fwd", "preference_loss_bwd", "preference_loss_step", "policy_loss_fwd",
                     "policy_loss_bwd", "policy_loss_step", "grad_norm_workspace", "grad_norm", "clip_grad_norm"}
    for n in names:
        assert hasattr(L, n), n


def test_version_and_status_strings(L):
    version = int(re.search(r"#define\s+FINETUNE_ABI_VERSION\s+(\d+)", open(HEADER).read()).group(1))
    assert L.finetune_abi_version() == version
    texts = {L.finetune_status_string(s) for s in range(8)}
    assert len(texts) == 8 and L.finetune_status_string(99) == b"unknown status"
    assert "strides" in str(bcl.FinetuneError("call", SHAPE)) and bcl.FinetuneError("call", SHAPE).status == SHAPE


A, B, C, D, E, W = (0x1000000 * k for k in range(1, 7))


def norm_fwd(L, x=A, w=B, b=None, y=C, mean=D, rstd=E, rows=4, d=64, xs=64, ys=64, eps=1e-5, dt=F32):
    return L.layer_norm_fwd(VP(x), VP(w), VP(b), VP(y), VP(mean), VP(rstd), I64(rows), I64(d), I64(xs), I64(ys),
                            F64(eps), INT(dt), None)


NORM_FWD = [
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None), OK), (dict(x=None), NULL), (dict(y=None), NULL),
    (dict(d=0), SIZE), (dict(d=-1), SIZE), (dict(d=(1 << 20) + 1), SIZE), (dict(rows=-1), SIZE),
    (dict(rows=1 << 31), SIZE), (dict(eps=-1.0), SIZE), (dict(eps=float("nan")), SIZE), (dict(eps=float("inf")), SIZE),
    (dict(xs=63), SHAPE), (dict(ys=63), SHAPE), (dict(xs=-64), SHAPE), (dict(xs=(1 << 63) - 1), SHAPE),
    (dict(dt=3), DTYPE), (dict(dt=-1), DTYPE), (dict(x=A + 2), ALIGN), (dict(x=A + 1, dt=BF16), ALIGN),
    (dict(w=B + 1), ALIGN), (dict(mean=D + 2), ALIGN), (dict(y=A + 64), ALIAS), (dict(y=A, ys=128), ALIAS),
    (dict(y=B), ALIAS), (dict(mean=A), ALIAS), (dict(rstd=D), ALIAS), (dict(mean=C + 1020), ALIAS),
    (dict(rstd=B + 252), ALIAS),
]


@pytest.mark.parametrize("change,want", NORM_FWD)
def test_layer_norm_fwd_arguments(L, change, want):
    assert norm_fwd(L, **change) == want


def norm_bwd(L, x=A, w=None, mean=D, rstd=E, dy=B, dx=C, dw=0x8000000, db=0x9000000, ws=W, ws_bytes=1 << 20, rows=4,
             d=64, xs=64, dys=64, dxs=64, dt=F32):
    return L.layer_norm_bwd(VP(x), VP(w), VP(mean), VP(rstd), VP(dy), VP(dx), VP(dw), VP(db), VP(ws), I64(ws_bytes),
                            I64(rows), I64(d), I64(xs), I64(dys), I64(dxs), INT(dt), None)


NORM_BWD = [
    (dict(rows=0, dw=None, db=None), OK), (dict(dx=None, dw=None, db=None), NULL), (dict(x=None), NULL),
    (dict(mean=None), NULL), (dict(rstd=None), NULL), (dict(dy=None), NULL), (dict(ws=None), NULL),
    (dict(ws_bytes=0), SIZE), (dict(ws_bytes=-1), SIZE), (dict(d=0), SIZE), (dict(rows=-3), SIZE),
    (dict(xs=1), SHAPE), (dict(dys=1), SHAPE), (dict(dxs=1), SHAPE), (dict(dt=7), DTYPE), (dict(dw=0x8000002), ALIGN),
    (dict(ws=W + 4), ALIGN), (dict(dx=B + 256), ALIAS), (dict(dx=B, dxs=65), ALIAS), (dict(dx=A), ALIAS),
    (dict(dw=A), ALIAS), (dict(db=0x8000000), ALIAS), (dict(ws=C), ALIAS), (dict(ws=A), ALIAS), (dict(dw=C), ALIAS),
    (dict(db=B + 512), ALIAS), (dict(rows=0, db=0x8000004), ALIAS),
]


@pytest.mark.parametrize("change,want", NORM_BWD)
def test_layer_norm_bwd_arguments(L, change, want):
    assert norm_bwd(L, **change) == want


def test_layer_norm_workspace(L):
    out = I64(-1)
    assert L.layer_norm_bwd_workspace(I64(4), I64(64), None) == NULL
    assert L.layer_norm_bwd_workspace(I64(4), I64(0), ctypes.byref(out)) == SIZE
    assert L.layer_norm_bwd_workspace(I64(-4), I64(8), ctypes.byref(out)) == SIZE
    assert L.layer_norm_bwd_workspace(I64(0), I64(64), ctypes.byref(out)) == OK and out.value == 0
    for rows, d in ((1, 1), (1000, 100), (70000, 4096), (3, 1 << 20)):
        assert L.layer_norm_bwd_workspace(I64(rows), I64(d), ctypes.byref(out)) == OK
        assert out.value >= 8 * d and out.value % 16 == 0


def logits(data=A, labels=B, seqs=2, positions=3, vocab=50, ss=150, ps=50, dt=F32):
    return Logits(data, labels, seqs, positions, vocab, ss, ps, dt)


LOGITS = [
    (dict(data=None), NULL), (dict(labels=None), NULL), (dict(seqs=-1), SIZE), (dict(positions=-1), SIZE),
    (dict(vocab=0), SIZE), (dict(vocab=(1 << 24) + 1), SIZE), (dict(seqs=1 << 16, positions=1 << 16), SIZE),
    (dict(ss=-1), SHAPE), (dict(ps=-50), SHAPE), (dict(ss=1 << 62), SHAPE), (dict(dt=3), DTYPE), (dict(dt=-1), DTYPE),
    (dict(data=A + 2), ALIGN), (dict(labels=B + 4), ALIGN),
]


def token_logprob(L, x, logp=C, lse=D, ws=W, ws_bytes=1 << 20):
    return L.token_logprob(ctypes.byref(x), VP(logp), VP(lse), VP(ws), I64(ws_bytes), None)


@pytest.mark.parametrize("change,want", LOGITS)
def test_logits_arguments(L, change, want):
    x, out = logits(**change), DLogits(E, 150, 50)
    how, pol = Preference(0, 0, 0.1, 0.0), Policy(0, 0, 0.2, 0.2, 0.0)
    assert token_logprob(L, x) == want
    assert L.token_logprob_bwd(ctypes.byref(x), VP(C), VP(D), ctypes.byref(out), None) == want
    small = [VP(0x10000000 + 0x10000 * k) for k in range(5)]
    assert L.preference_loss_fwd(ctypes.byref(x), VP(C), ctypes.byref(how), *small, VP(W), I64(1 << 20), None) == want
    assert L.policy_loss_fwd(ctypes.byref(x), VP(C), None, VP(D), ctypes.byref(pol), *small[:4], VP(W), I64(1 << 20),
                             None) == want


def test_token_logprob_arguments(L):
    assert L.token_logprob(None, VP(C), VP(D), VP(W), I64(1 << 20), None) == NULL
    assert token_logprob(L, logits(seqs=0)) == OK and token_logprob(L, logits(positions=0, data=None)) == OK
    assert token_logprob(L, logits(), logp=None) == NULL and token_logprob(L, logits(), ws_bytes=0) == SIZE
    assert token_logprob(L, logits(), ws=None) == NULL and token_logprob(L, logits(), ws=W + 8) == ALIGN
    assert token_logprob(L, logits(), lse=D + 1) == ALIGN and token_logprob(L, logits(), lse=C) == ALIAS
    assert token_logprob(L, logits(), logp=A) == ALIAS and token_logprob(L, logits(), logp=B + 8) == ALIAS
    assert token_logprob(L, logits(), ws=A) == ALIAS and token_logprob(L, logits(), ws=C) == ALIAS


DLOGITS = [
    (DLogits(None, 150, 50), NULL), (DLogits(E, 150, 49), SHAPE), (DLogits(E, 149, 50), SHAPE),
    (DLogits(E, -150, 50), SHAPE), (DLogits(E, 40, 100), SHAPE), (DLogits(E + 2, 150, 50), ALIGN),
    (DLogits(A, 151, 50), ALIAS), (DLogits(A + 200, 150, 50), ALIAS), (DLogits(B, 150, 50), ALIAS),
    (DLogits(C, 150, 50), ALIAS),
]


@pytest.mark.parametrize("out,want", DLOGITS)
def test_dlogits_arguments(L, out, want):
    x = logits()
    assert L.token_logprob_bwd(ctypes.byref(x), VP(C), VP(D), ctypes.byref(out), None) == want
    assert L.preference_loss_bwd(ctypes.byref(x), VP(C), VP(D), VP(W), ctypes.byref(out), None) == want
    assert L.policy_loss_bwd(ctypes.byref(x), VP(C), VP(D), VP(W), ctypes.byref(out), None) == want


def test_loss_parameters(L):
    x, out = logits(), DLogits(E, 150, 50)
    small = [VP(0x10000000 + 0x10000 * k) for k in range(5)]

    def preference(how, xx=x, ref=C):
        return L.preference_loss_fwd(ctypes.byref(xx), VP(ref), how and ctypes.byref(how), *small, VP(W), I64(1 << 20),
                                     None)

    assert preference(None) == NULL and preference(Preference(0, 0, 0.1, 0.0), ref=None) == NULL
    for bad in (Preference(3, 0, 0.1, 0.0), Preference(-1, 0, 0.1, 0.0), Preference(0, 0, 0.0, 0.0),
                Preference(0, 0, -1.0, 0.0), Preference(0, 0, float("nan"), 0.0), Preference(0, 0, 0.1, 0.5),
                Preference(0, 0, 0.1, -0.1), Preference(0, 0, float("inf"), 0.0)):
        assert preference(bad) == SIZE
    assert preference(Preference(0, 0, 0.1, 0.0), logits(seqs=3)) == SHAPE
    odd = logits(seqs=3)
    assert L.preference_loss_bwd(ctypes.byref(odd), VP(C), VP(D), VP(W), ctypes.byref(out), None) == SHAPE

    def policy(how, old=C, adv=D):
        return L.policy_loss_step(ctypes.byref(x), VP(old), None, VP(adv), how and ctypes.byref(how), F64(1.0),
                                  *small[:4], ctypes.byref(out), VP(W), I64(1 << 20), None)

    good = Policy(0, 0, 0.2, 0.2, 0.0)
    assert policy(None) == NULL and policy(good, old=None) == NULL and policy(good, adv=None) == NULL
    for bad in (Policy(3, 0, 0.2, 0.2, 0.0), Policy(-1, 0, 0.2, 0.2, 0.0), Policy(0, 0, -0.1, 0.2, 0.0),
                Policy(0, 0, 0.2, float("nan"), 0.0), Policy(0, 0, 0.2, 0.2, float("inf"))):
        assert policy(bad) == SIZE
    assert policy(good, old=0x10000000) == ALIAS and policy(good, adv=E) == ALIAS


def clip(L, tensors, max_norm=1.0, eps=1e-6, norm=D, ws=W, ws_bytes=1 << 20):
    t = (Tensor * len(tensors))(*tensors)
    return L.clip_grad_norm(t, I64(len(tensors)), F64(max_norm), F64(eps), VP(norm), VP(ws), I64(ws_bytes), None)


CLIP = [
    ([Tensor(None, A, 4, F32)], {}, NULL), ([Tensor(A, None, 4, F32)], {}, NULL), ([Tensor(A, A, 4, F32)], dict(norm=None), NULL),
    ([Tensor(A, A, 4, F32)], dict(ws=None), NULL), ([Tensor(A, A, 4, 3)], {}, DTYPE), ([Tensor(A, A, 4, -1)], {}, DTYPE),
    ([Tensor(A, A, -1, F32)], {}, SIZE), ([Tensor(A, A, (1 << 40) + 1, F32)], {}, SIZE),
    ([Tensor(A, A, 1 << 40, F32), Tensor(B, B, 1, F32)], {}, SIZE), ([Tensor(A, A, 4, F32)], dict(ws_bytes=0), SIZE),
    ([Tensor(A, A, 4, F32)], dict(max_norm=-1.0), SIZE), ([Tensor(A, A, 4, F32)], dict(max_norm=float("nan")), SIZE),
    ([Tensor(A, A, 4, F32)], dict(eps=-1.0), SIZE), ([Tensor(A + 2, A + 2, 4, F32)], {}, ALIGN),
    ([Tensor(A, B + 1, 4, BF16)], {}, ALIGN), ([Tensor(A, A, 4, F32)], dict(norm=D + 2), ALIGN),
    ([Tensor(A, A, 4, F32)], dict(ws=W + 8), ALIGN), ([Tensor(A, A + 8, 4, F32)], {}, ALIAS),
    ([Tensor(A, A, 4, F32), Tensor(A, A, 4, F32)], {}, ALIAS), ([Tensor(A, B, 4, F32), Tensor(B, C, 4, F32)], {}, ALIAS),
    ([Tensor(A, C, 4, F32), Tensor(B, C + 12, 4, F32)], {}, ALIAS), ([Tensor(B, B, 4, F32), Tensor(A, B + 4, 1, F32)], {}, ALIAS),
    ([Tensor(A, A, 4, F32)], dict(norm=A + 12), ALIAS), ([Tensor(A, A, 4, F32)], dict(ws=A), ALIAS),
    ([Tensor(A, B, 4, F32)], dict(norm=B), ALIAS), ([Tensor(A, A, 4, F32)], dict(norm=W), ALIAS),
]


@pytest.mark.parametrize("tensors,change,want", CLIP)
def test_clip_arguments(L, tensors, change, want):
    assert clip(L, tensors, **change) == want


def test_grad_norm_arguments(L):
    out = I64(-1)
    t = (Tensor * 1)(Tensor(A, None, 4, F32))
    assert L.grad_norm_workspace(None, I64(1), ctypes.byref(out)) == NULL and L.grad_norm_workspace(t, I64(1), None) == NULL
    assert L.grad_norm_workspace(t, I64(-1), ctypes.byref(out)) == SIZE
    assert L.grad_norm_workspace(t, I64(1), ctypes.byref(out)) == OK and out.value >= 8
    assert L.grad_norm(t, I64(1), None, VP(W), I64(64), None) == NULL
    assert L.grad_norm(t, I64(1), VP(D), VP(W), I64(0), None) == SIZE
    assert L.grad_norm(None, I64(2), VP(D), VP(W), I64(64), None) == NULL


def test_python_refusals():
    x = torch.zeros(2, 3, 8)
    lab = torch.zeros(2, 3, dtype=torch.int64)
    f = torch.zeros(2, 3)
    for call in (lambda: bcl.layer_norm_fwd(x), lambda: bcl.token_logprob(x, lab),
                 lambda: bcl.preference_loss_fwd(x, lab, f), lambda: bcl.policy_loss_step(x, lab, f, f),
                 lambda: bcl.clip_grad_norm([f], 1.0), lambda: bcl.grad_norm([]),
                 lambda: bcl.preference_loss_fwd(x, lab, f, kind="other"),
                 lambda: bcl.policy_loss_fwd(x, lab, f, f, reduction="other"),
                 lambda: bcl.layer_norm(x), lambda: bcl.token_logp(x, lab)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        bcl.clip_grad_norm([3.0], 1.0)


def _sanitized(kind, env):
    r = subprocess.run([build_emu.build(kind), "small"], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, **env))
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[:4000]
    assert re.match(r"ok 28 \d+\n", r.stdout), r.stdout


def test_kernels_on_cpu_threads_address_sanitizer():
    _sanitized("asan", {"ASAN_OPTIONS": "detect_leaks=0"})


def test_kernels_on_cpu_threads_thread_sanitizer():
    _sanitized("tsan", {})


def test_no_kernel_uses_scratch(L):
    kernels = build.kernel_resources(build.FINETUNE_LIB)
    for family in ("layer_norm_fwd", "layer_norm_bwd", "layer_norm_wide_fwd", "token_logprob", "logits_grad",
                   "preference_kernel", "policy_kernel", "policy_step", "grad_square", "grad_scale"):
        assert any(family in k for k in kernels), family
    # (scalar registers saved in lanes of a vector register take no memory)
    bad = {k: r for k, r in kernels.items()
           if r["private_segment_fixed_size"] or r["vgpr_spill_count"] or r["uses_dynamic_stack"]}
    assert not bad, sorted(bad)
