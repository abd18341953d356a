"""CPU checks of the sublayer operators: the C ABI's exports and argument
checks, the Python calls' refusals, and the code object.

The pointers of the ABI cases are fake and never dereferenced: every call
carries an invalid argument or asks for no work, so no kernel is enqueued."""

from __future__ import annotations

import ctypes
import glob
import os
import re

import pytest
import torch

import block_circulant_layers_amd as bcl
from block_circulant_layers_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "attention.h")
I64, F64, INT, VP, U64 = ctypes.c_int64, ctypes.c_double, ctypes.c_int, ctypes.c_void_p, ctypes.c_uint64
OK, NULL, SIZE, SHAPE, DTYPE, ALIGN, ALIAS = range(7)
F32, BF16, F16 = 0, 1, 2


class Buckets(ctypes.Structure):
    _fields_ = [("count", I64), ("max_distance", I64), ("two_sided", I64)]


class Problem(ctypes.Structure):
    _fields_ = [("batch", I64), ("queries", I64), ("keys", I64), ("heads", I64), ("kv_heads", I64), ("head_dim", I64),
                ("dtype", I64), ("scale", F64), ("causal", I64), ("key_begin", VP), ("key_end", VP), ("bias", VP),
                ("buckets", Buckets)]


class Tensor(ctypes.Structure):
    _fields_ = [("data", VP), ("batch_stride", I64), ("token_stride", I64), ("head_stride", I64)]


class Dropout(ctypes.Structure):
    _fields_ = [("p", F64), ("seed", U64), ("offset", U64), ("device_seed", VP)]


@pytest.fixture(scope="module")
def L():
    sources = glob.glob(os.path.join(build.CSRC, "finetune", "*")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    newest = max(os.path.getmtime(s) for s in sources)
    if any(not os.path.exists(p) or os.path.getmtime(p) < newest for p in (build.FINETUNE_LIB, build.FINETUNE_HOST)):
        build.build_finetune(verbose=False)
    return ctypes.CDLL(build.FINETUNE_LIB)


def test_exports_every_declared_symbol(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(\w+)\s*\(", src, flags=re.M))
    assert names == {"attention_abi_version", "relative_bias_fwd", "relative_bias_workspace", "relative_bias_bwd",
                     "attention_workspace", "attention_fwd", "attention_bwd", "dropout_fwd", "dropout_bwd"}
    for n in names:
        assert hasattr(L, n), n
    version = int(re.search(r"#define\s+ATTENTION_ABI_VERSION\s+(\d+)", open(HEADER).read()).group(1))
    assert L.attention_abi_version() == version


# far apart, so that no two overlap unless a case says so
Q, K, V, O, DO, DQ, DK, DV, LSE, WS, TABLE, DTABLE, LO, HI = (0x10000000 * n for n in range(1, 15))
BATCH, TQ, TK, HEADS, KV, DIM = 2, 5, 7, 4, 2, 8


def problem(**change):
    base = dict(batch=BATCH, queries=TQ, keys=TK, heads=HEADS, kv_heads=KV, head_dim=DIM, dtype=F32, scale=0.5,
                causal=0, key_begin=None, key_end=None, bias=None, buckets=Buckets(8, 20, 1))
    return Problem(**(base | change))


def tensor(p, tokens, heads, **change):
    base = dict(data=p, batch_stride=tokens * heads * DIM, token_stride=heads * DIM, head_stride=DIM)
    return Tensor(**(base | change))


def tensors(**change):
    t = {n: tensor(p, TQ, HEADS) for n, p in (("q", Q), ("o", O), ("dout", DO), ("dq", DQ))}
    t |= {n: tensor(p, TK, KV) for n, p in (("k", K), ("v", V), ("dk", DK), ("dv", DV))}
    return t | change


def fwd(L, a=None, lse=LSE, ws=WS, ws_bytes=1 << 24, **change):
    a, t = a or problem(), tensors(**change)
    ref = [t[n] and ctypes.byref(t[n]) for n in "qkvo"]
    return L.attention_fwd(ctypes.byref(a), *ref, VP(lse), VP(ws), I64(ws_bytes), None)


def bwd(L, a=None, lse=LSE, dbias=None, ws=WS, ws_bytes=1 << 24, **change):
    a, t = a or problem(), tensors(**change)
    r = {n: x and ctypes.byref(x) for n, x in t.items()}
    return L.attention_bwd(ctypes.byref(a), r["q"], r["k"], r["v"], r["o"], VP(lse), r["dout"], r["dq"], r["dk"],
                           r["dv"], VP(dbias), VP(ws), I64(ws_bytes), None)


PROBLEMS = [
    (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE), (dict(batch=-1), SIZE), (dict(queries=-1), SIZE),
    (dict(keys=-1), SIZE), (dict(keys=(1 << 24) + 1), SIZE), (dict(heads=0), SIZE), (dict(kv_heads=0), SIZE),
    (dict(head_dim=0), SIZE), (dict(head_dim=129), SIZE), (dict(heads=3), SHAPE), (dict(kv_heads=8), SHAPE),
    (dict(scale=0.0), SIZE), (dict(scale=-1.0), SIZE), (dict(scale=float("nan")), SIZE),
    (dict(scale=float("inf")), SIZE), (dict(scale=1e39), SIZE), (dict(scale=1e-60), SIZE),
    (dict(key_begin=LO + 2), ALIGN), (dict(key_end=HI + 1), ALIGN), (dict(bias=TABLE + 2), ALIGN),
    (dict(bias=TABLE, buckets=Buckets(7, 20, 1)), SIZE), (dict(bias=TABLE, buckets=Buckets(1, 20, 0)), SIZE),
    (dict(bias=TABLE, buckets=Buckets(2, 20, 1)), SIZE), (dict(bias=TABLE, buckets=Buckets(257, 500, 0)), SIZE),
    (dict(bias=TABLE, buckets=Buckets(514, 500, 1)), SIZE), (dict(bias=TABLE, buckets=Buckets(8, 2, 1)), SIZE),
    (dict(bias=TABLE, buckets=Buckets(8, 1025, 1)), SIZE), (dict(bias=TABLE, buckets=Buckets(-8, 20, 1)), SIZE),
    (dict(batch=1 << 20, heads=64, kv_heads=64), SIZE),
    (dict(batch=1, queries=1, keys=1, heads=1 << 22, bias=TABLE), SIZE),
    (dict(batch=1 << 18, heads=64, kv_heads=64, queries=1 << 24, keys=1), SIZE),
]


@pytest.mark.parametrize("change,want", PROBLEMS)
def test_problem(L, change, want):
    a, out = problem(**change), I64(-1)
    for backward in (0, 1):
        assert L.attention_workspace(ctypes.byref(a), INT(backward), ctypes.byref(out)) == want
    assert fwd(L, a) == want and bwd(L, a) == want


def test_workspace(L):
    a, out = problem(), I64(-1)
    assert L.attention_workspace(None, INT(0), ctypes.byref(out)) == NULL
    assert L.attention_workspace(ctypes.byref(a), INT(0), None) == NULL
    assert L.attention_workspace(ctypes.byref(a), INT(0), ctypes.byref(out)) == OK and out.value >= 0
    assert L.attention_workspace(ctypes.byref(a), INT(1), ctypes.byref(out)) == OK
    assert out.value >= BATCH * TQ * HEADS * 4 and out.value % 16 == 0


def queries(p, **change):
    return tensor(p, TQ, HEADS, **change)


def keys(p, **change):
    return tensor(p, TK, KV, **change)


FUSED = dict(token_stride=(HEADS + 2 * KV) * DIM, head_stride=DIM)
Q_BYTES, TOKEN = BATCH * TQ * HEADS * DIM * 4, HEADS * DIM * 4

FWD = [
    (dict(q=None), NULL), (dict(o=None), NULL), (dict(q=queries(None)), NULL), (dict(k=keys(None)), NULL),
    (dict(v=keys(None)), NULL), (dict(o=queries(None)), NULL), (dict(lse=None), NULL), (dict(lse=LSE + 2), ALIGN),
    (dict(q=queries(Q + 2)), ALIGN), (dict(o=queries(O + 1)), ALIGN), (dict(q=queries(Q, token_stride=-1)), SHAPE),
    (dict(k=keys(K, batch_stride=1 << 62)), SHAPE), (dict(o=queries(O, head_stride=DIM - 1)), SHAPE),
    (dict(o=queries(O, batch_stride=0)), SHAPE), (dict(o=queries(O, token_stride=DIM)), SHAPE),
    (dict(o=queries(Q)), ALIAS), (dict(o=queries(K)), ALIAS), (dict(o=queries(V + 16)), ALIAS),
    (dict(o=queries(Q + Q_BYTES - 4)), ALIAS), (dict(lse=Q), ALIAS), (dict(lse=O + 8), ALIAS),
    (dict(q=queries(Q, token_stride=2 * HEADS * DIM, batch_stride=2 * TQ * HEADS * DIM),
          o=queries(Q + TOKEN - 4, token_stride=2 * HEADS * DIM, batch_stride=2 * TQ * HEADS * DIM)), ALIAS),
]


@pytest.mark.parametrize("change,want", FWD)
def test_attention_fwd_arguments(L, change, want):
    assert fwd(L, **change) == want


def test_attention_no_work(L):
    for change in (dict(batch=0), dict(queries=0)):
        assert fwd(L, problem(**change), lse=None, q=queries(None), o=queries(None)) == OK
    assert bwd(L, problem(batch=0), lse=None, ws=None, ws_bytes=0) == OK
    a = problem(queries=1, keys=4096)  # split: a workspace is needed
    assert fwd(L, a, ws=None) == NULL and fwd(L, a, ws_bytes=0) == SIZE and fwd(L, a, ws=WS + 4) == ALIGN
    assert fwd(L, a, ws=Q) == ALIAS and fwd(L, a, ws=LSE) == ALIAS and fwd(L, a, ws=O) == ALIAS
    for bad in (dict(key_end=O), dict(key_begin=LSE), dict(bias=O + 64)):
        assert fwd(L, problem(**bad)) == ALIAS


BWD = [
    (dict(dout=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dv=None), NULL),
    (dict(dout=queries(None)), NULL), (dict(dq=queries(None)), NULL), (dict(lse=None), NULL), (dict(ws=None), NULL),
    (dict(ws_bytes=0), SIZE), (dict(ws=WS + 8), ALIGN), (dict(dbias=DTABLE), SHAPE), (dict(dq=queries(DQ + 2)), ALIGN),
    (dict(lse=LSE + 1), ALIGN), (dict(dk=keys(DK, head_stride=0)), SHAPE), (dict(dv=keys(DV, token_stride=0)), SHAPE),
    (dict(dout=queries(DO, head_stride=-8)), SHAPE), (dict(dq=queries(Q)), ALIAS), (dict(dq=queries(DO)), ALIAS),
    (dict(dk=keys(K)), ALIAS), (dict(dv=keys(DK)), ALIAS), (dict(dv=keys(DK + 4)), ALIAS), (dict(dk=keys(LSE)), ALIAS),
    (dict(dq=queries(O)), ALIAS), (dict(ws=DQ), ALIAS), (dict(ws=V), ALIAS), (dict(ws=LSE), ALIAS),
]


@pytest.mark.parametrize("change,want", BWD)
def test_attention_bwd_arguments(L, change, want):
    assert bwd(L, **change) == want


def test_attention_bwd_bias_and_fused_buffers(L):
    a = problem(bias=TABLE)
    for at, want in ((TABLE, ALIAS), (DTABLE + 2, ALIGN), (WS + 16, ALIAS), (DQ, ALIAS), (Q, ALIAS), (LSE, ALIAS)):
        assert bwd(L, a, dbias=at) == want
    # gradients that interleave in one buffer are apart; shifted by one head they are not
    n = (HEADS + 2 * KV) * DIM
    part = {"dq": (0, TQ), "dk": (HEADS, TK), "dv": (HEADS + KV, TK)}

    def fused(shift):
        return {name: Tensor(DQ + 4 * DIM * (h + (shift if name == "dv" else 0)), TK * n, n, DIM)
                for name, (h, _) in part.items()}

    apart, over = fused(0), fused(-1)
    assert bwd(L, **apart, ws=None) == NULL  # the overlap check comes after the workspace's
    assert bwd(L, **over) == ALIAS
    odd = fused(0)
    odd["dv"].batch_stride += DIM  # sequences not a whole number of tokens apart
    assert bwd(L, **odd) == ALIAS


def bias_fwd(L, table=TABLE, bias=O, heads=4, tq=5, tk=7, b=Buckets(8, 20, 1), dt=F32):
    return L.relative_bias_fwd(VP(table), VP(bias), I64(heads), I64(tq), I64(tk), b and ctypes.byref(b), INT(dt), None)


BIAS_FWD = [
    (dict(tq=0), OK), (dict(tk=0, table=None, bias=None), OK), (dict(table=None), NULL), (dict(bias=None), NULL),
    (dict(b=None), NULL), (dict(b=Buckets(9, 20, 1)), SIZE), (dict(b=Buckets(8, 2000, 0)), SIZE), (dict(heads=0), SIZE),
    (dict(tq=-1), SIZE), (dict(tk=1 << 25), SIZE), (dict(dt=5), DTYPE), (dict(table=TABLE + 2), ALIGN),
    (dict(bias=O + 1, dt=BF16), ALIGN), (dict(bias=TABLE + 64), ALIAS), (dict(tq=1 << 24, tk=1 << 24), SIZE),
]


@pytest.mark.parametrize("change,want", BIAS_FWD)
def test_relative_bias_fwd_arguments(L, change, want):
    assert bias_fwd(L, **change) == want


def bias_bwd(L, dbias=DO, sb=140, sh=35, sq=7, dtable=DTABLE, batch=2, heads=4, tq=5, tk=7, b=Buckets(8, 20, 1), ws=WS,
             ws_bytes=1 << 20, dt=F32):
    return L.relative_bias_bwd(VP(dbias), I64(sb), I64(sh), I64(sq), VP(dtable), I64(batch), I64(heads), I64(tq),
                               I64(tk), b and ctypes.byref(b), VP(ws), I64(ws_bytes), INT(dt), None)


BIAS_BWD = [
    (dict(dbias=None), NULL), (dict(dtable=None), NULL), (dict(b=None), NULL), (dict(ws=None), NULL),
    (dict(ws_bytes=0), SIZE), (dict(ws=WS + 8), ALIGN), (dict(dt=3), DTYPE), (dict(batch=-1), SIZE),
    (dict(heads=0), SIZE), (dict(sb=-1), SHAPE), (dict(sq=1 << 62), SHAPE), (dict(dbias=DO + 2), ALIGN),
    (dict(dtable=DTABLE + 1), ALIGN), (dict(dtable=DO + 8), ALIAS), (dict(ws=DO), ALIAS), (dict(ws=DTABLE), ALIAS),
    (dict(b=Buckets(8, 0, 1)), SIZE),
]


@pytest.mark.parametrize("change,want", BIAS_BWD)
def test_relative_bias_bwd_arguments(L, change, want):
    assert bias_bwd(L, **change) == want


def drop(L, x=Q, res=None, y=O, rows=4, d=8, xs=8, rs=8, ys=8, p=0.1, seed=None, dt=F32):
    how = Dropout(p, 3, 4, seed)
    return L.dropout_fwd(VP(x), VP(res), VP(y), I64(rows), I64(d), I64(xs), I64(rs), I64(ys), ctypes.byref(how),
                         INT(dt), None)


DROP = [
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None), OK), (dict(x=None), NULL), (dict(y=None), NULL),
    (dict(p=-0.1), SIZE), (dict(p=1.1), SIZE), (dict(p=float("nan")), SIZE), (dict(d=0), SIZE), (dict(rows=-1), SIZE),
    (dict(rows=1 << 40), SIZE), (dict(xs=7), SHAPE), (dict(ys=-8), SHAPE), (dict(res=K, rs=7), SHAPE),
    (dict(dt=3), DTYPE), (dict(x=Q + 2), ALIGN), (dict(res=K + 1), ALIGN), (dict(seed=LO + 4), ALIGN),
    (dict(y=Q + 4), ALIAS), (dict(y=Q, ys=9), ALIAS), (dict(res=O + 8), ALIAS), (dict(res=O, rs=9), ALIAS),
    (dict(seed=O + 8), ALIAS),
]


@pytest.mark.parametrize("change,want", DROP)
def test_dropout_arguments(L, change, want):
    assert drop(L, **change) == want
    assert L.dropout_fwd(VP(Q), None, VP(O), I64(1), I64(8), I64(8), I64(8), I64(8), None, INT(0), None) == NULL
    how = Dropout(2.0, 3, 4, None)
    assert L.dropout_bwd(VP(Q), VP(O), I64(1), I64(8), I64(8), I64(8), ctypes.byref(how), INT(0), None) == SIZE


def test_python_refusals():
    x, table = torch.zeros(1, 2, 3, 8), torch.zeros(8, 3)
    for call in (lambda: bcl.attention_fwd(x, x, x), lambda: bcl.attention_bwd(x, x, x, x, x[..., 0], x),
                 lambda: bcl.attention(x, x, x), lambda: bcl.relative_bias_fwd(table, 2, 2),
                 lambda: bcl.relative_bias_bwd(x, 8), lambda: bcl.relative_bias(table, 2, 2),
                 lambda: bcl.dropout_fwd(x, 0.1, 1), lambda: bcl.dropout_bwd(x, 0.1, 1), lambda: bcl.dropout(x, 0.1),
                 lambda: bcl.Dropout(1.5)):
        with pytest.raises(ValueError):
            call()
    for seed in (-1, 1 << 64, 0.5, "x"):
        with pytest.raises(TypeError):
            bcl.dropout_fwd(x, 0.1, seed)
    assert bcl.Dropout(0.3).eval()(x) is x and torch.equal(bcl.Dropout(0.0)(x, residual=x + 1), x + 1)


def test_no_kernel_uses_scratch(L):
    kernels = build.kernel_resources(build.FINETUNE_LIB)
    for family in ("attention_fwd_kernel", "attention_join", "attention_dq", "attention_dkv", "attention_sum",
                   "relative_bias_fwd", "relative_bias_bwd", "bias_parts", "dropout_kernel", "dropout_rows"):
        assert any(family in k for k in kernels), family
    bad = {k: r for k, r in kernels.items()
           if r["private_segment_fixed_size"] or r["vgpr_spill_count"] or r["uses_dynamic_stack"]}
    assert not bad, sorted(bad)
