"""GPU parity of attention, relative position bias and dropout against the float64 oracle.

Bounds come from tests/attention_util.py: the worst case of the kernels'
arithmetic plus the roundings to storage.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import block_circulant_layers_amd as bcl
from tests import attention_util as au
from tests.attention_util import DEV, U, ao, f64, rng, store_err, stored
from tests.finetune_util import TORCH, within

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16", "f16"]

# batch, queries, keys, heads, key heads, head size
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 5, 7, 2, 1, 8), (1, 64, 64, 4, 2, 16), (2, 33, 65, 3, 3, 33), (1, 129, 127, 2, 2, 64),
          (1, 200, 130, 4, 1, 80), (1, 70, 300, 2, 2, 128), (2, 1, 513, 8, 2, 64), (3, 17, 700, 4, 4, 40),
          (1, 300, 300, 2, 1, 96), (1, 257, 31, 1, 1, 127)]
MODES = {"plain": {}, "causal": dict(causal=True), "spans": dict(spanned=True),
         "both": dict(causal=True, spanned=True), "bias": dict(table=8),
         "bias_one_sided": dict(table=7, two_sided=False, causal=True, spanned=True)}


def check(shape, dtype, mode, key=0, **more):
    b, tq, tk, hq, hk, d = shape
    how = MODES[mode] | more
    x, kw, see, bias = au.case((key, *shape), *shape, dtype, **how)
    (q, qr), (k, kr), (v, vr), (do, dr) = (x[n] for n in ("q", "k", "v", "dout"))
    want, lse, p = ao.attention(qr, kr, vr, kw["scale"], see, bias)
    o, got_lse = bcl.attention_fwd(q, k, v, **kw)
    bo, bl = au.forward_bounds(qr, kr, vr, kw["scale"], want, lse, p, dtype, bias)
    within(f64(got_lse), lse, bl)
    within(f64(o), want, bo)
    dq, dk, dv, dbias = bcl.attention_bwd(q, k, v, o, got_lse, do, **kw)
    gq, gk, gv, ds = ao.attention_bwd(qr, kr, vr, p, dr, kw["scale"])
    bq, bk, bv, e_ds = au.backward_bounds(qr, kr, vr, dr, kw["scale"], want, lse, p, ds, bo, (gq, gk, gv), dtype, bias)
    within(f64(dv), gv, bv)
    within(f64(dk), gk, bk)
    within(f64(dq), gq, bq)
    if bias is None:
        assert dbias is None
        return
    count = kw["bias"].shape[0]
    total = ao.relative_bias_bwd(ds, count, kw["max_distance"], kw["bidirectional"])
    e = ao.relative_bias_bwd(e_ds + (tq + 64) * U * np.abs(ds), count, kw["max_distance"], kw["bidirectional"])
    within(f64(dbias), total, e + 2 * U * np.abs(total) + 1e-30)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_attention(shape, dtype, mode):
    check(shape, dtype, mode)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_more_queries_than_keys(dtype):
    # a causal mask leaves the first queries without a key
    check((2, 150, 70, 2, 2, 32), dtype, "causal")
    check((2, 90, 10, 4, 2, 24), dtype, "both")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale,spread", [(3.0, 1.0), (1e-3, 1.0), (0.1, 8.0)])
def test_attention_peaked_and_flat(dtype, scale, spread):
    check((1, 100, 90, 2, 1, 64), dtype, "causal", scale=scale, spread=spread)


@pytest.mark.parametrize("table,distance,two_sided", [(4, 3, True), (2, 1024, False), (512, 1024, True), (64, 300, True),
                                                      (31, 128, False)])
def test_attention_bias_buckets(table, distance, two_sided):
    check((1, 350, 420, 2, 2, 32), "f32", "bias", table=table, distance=distance, two_sided=two_sided)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_bias_at_the_largest_lds(dtype):
    check((1, 90, 140, 2, 1, 128), dtype, "bias", table=512, distance=1024)


def test_attention_bias_of_shared_heads():
    check((2, 70, 90, 4, 2, 32), "bf16", "bias")
    check((1, 1, 600, 8, 2, 64), "f32", "bias_one_sided")


@pytest.mark.parametrize("power", [-12, -6, 6, 12])
def test_half_gradients_of_any_size(power):
    """Gradients far from 1 lose no bits on the way; dout grows along the queries, so the kernels rescale."""
    shape = (1, 200, 150, 2, 1, 64)
    x, kw, see, _ = au.case((5,), *shape, "f16")
    (q, qr), (k, kr), (v, vr), (do, _) = (x[n] for n in ("q", "k", "v", "dout"))
    grow = torch.linspace(0, 1, 200, device=DEV)[None, :, None, None]
    do = (do.float() * torch.exp2(power * grow)).half()
    dr = f64(do)
    o, lse = bcl.attention_fwd(q, k, v, **kw)
    _, _, p = ao.attention(qr, kr, vr, kw["scale"], see)
    got = bcl.attention_bwd(q, k, v, o, lse, do, **kw)
    want = ao.attention_bwd(qr, kr, vr, p, dr, kw["scale"])
    for a, b in zip(got[:3], want[:3]):
        # normwise: three roundings to half (o, ds or p, the result) at 2^-11 each, and sums of unlike signs
        assert np.linalg.norm(f64(a) - b) <= 4 * 2.0**-11 * np.linalg.norm(b) + 2.0**-24 * np.sqrt(b.size)


def test_attention_gradient_against_differences():
    """fp32 gradients against differences of the float64 forward along random directions."""
    shape = (2, 40, 50, 4, 2, 32)
    x, kw, see, _ = au.case((6,), *shape, "f32", table=8, spanned=True)
    refs = [x[n][1] for n in ("q", "k", "v")] + [f64(kw["bias"])]
    up = x["dout"][1]
    o, lse = bcl.attention_fwd(*(x[n][0] for n in "qkv"), **kw)
    grads = bcl.attention_bwd(*(x[n][0] for n in "qkv"), o, lse, x["dout"][0], **kw)

    def loss(a):
        bias = ao.relative_bias(a[3], 40, 50, kw["max_distance"], True)
        return (ao.attention(*a[:3], kw["scale"], see, bias)[0] * up).sum()

    for n, g in enumerate(grads):
        direction = rng(6, n).standard_normal(refs[n].shape)
        hi, lo = list(refs), list(refs)
        hi[n], lo[n] = refs[n] + 1e-5 * direction, refs[n] - 1e-5 * direction
        slope = (loss(hi) - loss(lo)) / 2e-5
        scale = np.linalg.norm(f64(g)) * np.linalg.norm(direction)
        assert abs(slope - (f64(g) * direction).sum()) <= 1e-5 * scale


# ---------------------------------------------------------------------------
# layouts, edges, calling
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 24, 13])
def test_attention_strides(dtype, d):
    """Parts of a fused projection, heads before tokens, an odd first element; gradients into a fused buffer."""
    b, t, hq, hk = 2, 75, 4, 2
    r = rng(8, d)
    fused, _ = stored(r.standard_normal((b, t, (hq + 2 * hk) * d + 3)), dtype)
    fused = fused.to(DEV)[:, :, 3:].unflatten(2, (hq + 2 * hk, d))
    q, k, v = fused[:, :, :hq], fused[:, :, hq:hq + hk], fused[:, :, hq + hk:]
    do = stored(r.standard_normal((b, hq, t, d)), dtype)[0].to(DEV).transpose(1, 2)
    plain = [x.contiguous() for x in (q, k, v)]
    o0, lse0 = bcl.attention_fwd(*plain, causal=True)
    out = torch.full((b, hq, t, d), 7.0, device=DEV, dtype=TORCH[dtype]).transpose(1, 2)
    o, lse = bcl.attention_fwd(q, k, v, causal=True, o=out)
    assert o is out and torch.equal(o, o0) and torch.equal(lse, lse0)
    want = bcl.attention_bwd(*plain, o0, lse0, do.contiguous(), causal=True)
    buffer = torch.full((b, t, (hq + 2 * hk) * d + 3), 7.0, device=DEV, dtype=TORCH[dtype])
    grad = buffer[:, :, 3:].unflatten(2, (hq + 2 * hk, d))
    parts = grad[:, :, :hq], grad[:, :, hq:hq + hk], grad[:, :, hq + hk:]
    got = bcl.attention_bwd(q, k, v, o, lse, do, causal=True, dq=parts[0], dk=parts[1], dv=parts[2])
    for a, w, part in zip(got, want, parts):
        assert a is part and torch.equal(a, w)
    assert (buffer[:, :, :3] == 7.0).all()
    # keys and values shared by the whole batch
    one = bcl.attention_fwd(q, k[:1].expand(b, -1, -1, -1), v[:1].expand(b, -1, -1, -1))[0]
    assert torch.equal(one, bcl.attention_fwd(q.contiguous(), k[:1].repeat(b, 1, 1, 1), v[:1].repeat(b, 1, 1, 1))[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries", [1, 90])
def test_attention_reads_no_masked_key(dtype, queries):
    """Whatever stands outside a span, and in dout of queries without a key, changes nothing."""
    b, tk, hq, hk, d = 3, 200, 4, 2, 40
    x, kw, _, _ = au.case((9, queries), b, queries, tk, hq, hk, d, dtype, spanned=True, causal=True)
    q, k, v, do = (x[n][0] for n in ("q", "k", "v", "dout"))
    o0, lse0 = bcl.attention_fwd(q, k, v, **kw)
    g0 = bcl.attention_bwd(q, k, v, o0, lse0, do, **kw)
    j = torch.arange(tk, device=DEV)
    out = ((j < kw["key_begin"][:, None]) | (j >= kw["key_end"][:, None]))[:, :, None, None]
    for bad in (float("nan"), float("inf"), torch.finfo(TORCH[dtype]).min):
        k2, v2 = torch.where(out, bad, k), torch.where(out, bad, v)
        do2, q2 = (torch.where((lse0 == -torch.inf).transpose(1, 2)[..., None], bad, t) for t in (do, q))
        o, lse = bcl.attention_fwd(q2, k2, v2, **kw)
        assert torch.equal(o, o0) and torch.equal(lse, lse0)
        for a, w in zip(bcl.attention_bwd(q2, k2, v2, o, lse, do2, **kw)[:3], g0):
            assert torch.equal(a, w)
    assert (lse0[-1] == -torch.inf).all() and not o0[-1].any() and not g0[0][-1].any() and not g0[1][-1].any()


def test_attention_spans_are_clamped():
    """Ends past the keys, negative begins, ends before begins."""
    x, kw, _, _ = au.case((15,), 4, 70, 90, 2, 1, 32, "bf16")
    q, k, v, do = (x[n][0] for n in ("q", "k", "v", "dout"))

    def both(begin, end):
        spans = dict(key_begin=torch.tensor(begin, device=DEV, dtype=torch.int32),
                     key_end=torch.tensor(end, device=DEV, dtype=torch.int32))
        o, lse = bcl.attention_fwd(q, k, v, **kw, **spans)
        return [o, lse, *bcl.attention_bwd(q, k, v, o, lse, do, **kw, **spans)[:3]]

    big = (1 << 31) - 1
    for a, b in zip(both([-5, 10, 60, big], [big, 50, 20, big]), both([0, 10, 60, 90], [90, 50, 60, 90])):
        assert torch.equal(a, b)


def test_attention_bias_of_minus_infinity():
    """A bucket that is ruled out takes no part; a query left with such buckets alone sees no key."""
    x, kw, see, bias = au.case((16,), 1, 60, 60, 2, 2, 32, "f32", table=7, two_sided=False, causal=True)
    q, k, v, do = (x[n][0] for n in ("q", "k", "v", "dout"))
    kw["bias"][0] = -torch.inf  # a query's own position: the first query has no other
    where = ao.bucket_matrix(60, 60, 7, kw["max_distance"], False)
    see = see & (where != 0)
    o, lse = bcl.attention_fwd(q, k, v, **kw)
    want, want_lse, p = ao.attention(*(x[n][1] for n in "qkv"), kw["scale"], see, bias)
    bo, bl = au.forward_bounds(*(x[n][1] for n in "qkv"), kw["scale"], want, want_lse, p, "f32", bias)
    within(f64(o), want, bo)
    within(f64(lse), want_lse, bl)
    grads = bcl.attention_bwd(q, k, v, o, lse, do, **kw)
    for got, exact in zip(grads[:3], ao.attention_bwd(*(x[n][1] for n in "qkv"), p, x["dout"][1], kw["scale"])):
        # fp32 throughout, sums of at most 60 terms of either sign
        assert np.linalg.norm(f64(got) - exact) <= 1e-5 * np.linalg.norm(exact)
    assert not grads[3][0].any() and grads[3].isfinite().all() and not o[0, 0].any()


@pytest.mark.parametrize("tk", [40, 900])
def test_queries_without_keys_stay_zero_beside_infinities(tk):
    """Causal, more queries than keys: the first ones see none, whatever the keys hold that others see."""
    x, kw, _, _ = au.case((17, tk), 1, tk + 20, tk, 2, 2, 32, "bf16", causal=True)
    q, k, v, do = (x[n][0] for n in ("q", "k", "v", "dout"))
    v[0, 0] = torch.inf
    k[0, 1] = torch.nan
    o, lse = bcl.attention_fwd(q, k, v, **kw)
    assert not o[:, :20].any() and (lse[:, :, :20] == -torch.inf).all()
    dq = bcl.attention_bwd(q, k, v, o, lse, do, **kw)[0]
    assert not dq[:, :20].any()


@pytest.mark.parametrize("bias", [False, True])
def test_attention_of_nothing(bias):
    kw = dict(bias=torch.ones(8, 2, device=DEV)) if bias else {}

    def new(b, t, h=2):
        return torch.ones(b, t, h, 16, device=DEV)

    for b, tq, tk in ((0, 3, 4), (2, 0, 4), (2, 3, 0)):
        q, k = new(b, tq), new(b, tk)
        o, lse = bcl.attention_fwd(q, k, k, **kw)
        assert o.shape == q.shape and not o.any() and (lse == -torch.inf).all() and lse.shape == (b, 2, tq)
        dq, dk, dv, dbias = bcl.attention_bwd(q, k, k, o, lse, q, **kw)
        assert not dq.any() and not dk.any() and not dv.any() and (dbias is None or not dbias.any())
        assert (dbias is not None) == bias


def test_attention_of_infinite_scores():
    """A NaN or an infinite score stays in its own row."""
    x, kw, _, _ = au.case((10,), 1, 70, 90, 2, 2, 32, "f32")
    q, k, v = (x[n][0] for n in "qkv")
    o0, lse0 = bcl.attention_fwd(q, k, v, **kw)
    q = q.clone()
    q[0, 3, 1, 0] = float("nan")
    o, lse = bcl.attention_fwd(q, k, v, **kw)
    assert o[0, 3, 1].isnan().all() and lse[0, 1, 3].isnan()
    keep = torch.ones(70, dtype=torch.bool, device=DEV)
    keep[3] = False
    assert torch.equal(o[:, keep], o0[:, keep]) and torch.equal(o[0, 3, 0], o0[0, 3, 0])


@pytest.mark.parametrize("dtype", ["bf16"])
def test_attention_offsets_past_32_bits(dtype):
    """Keys whose last rows lie beyond 2^31 elements and 2^32 bytes."""
    tk, hk, d, st = 70, 1, 32, 1 << 25
    r = rng(11)
    buffer = torch.empty((tk - 1) * st + 4 * d, device=DEV, dtype=TORCH[dtype])
    k, v, dk, dv = (buffer[n * d:].as_strided((1, tk, hk, d), (0, st, d, 1)) for n in range(4))
    kd, vd = (stored(r.standard_normal((1, tk, hk, d)), dtype)[0].to(DEV) for _ in range(2))
    k.copy_(kd), v.copy_(vd)
    q, do = (stored(r.standard_normal((1, 80, 2, d)), dtype)[0].to(DEV) for _ in range(2))
    o0, lse0 = bcl.attention_fwd(q, kd, vd)
    o, lse = bcl.attention_fwd(q, k, v)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    want = bcl.attention_bwd(q, kd, vd, o, lse, do)
    got = bcl.attention_bwd(q, k, v, o, lse, do, dk=dk, dv=dv)
    for a, w in zip(got[:3], want[:3]):
        assert torch.equal(a, w)


@pytest.mark.parametrize("shape", [(2, 300, 310, 4, 2, 64), (1, 3, 900, 8, 2, 64)])
def test_attention_repeats_bitwise(shape):
    x, kw, _, _ = au.case((12,), *shape, "bf16", table=32)
    q, k, v, do = (x[n][0] for n in ("q", "k", "v", "dout"))
    o, lse = bcl.attention_fwd(q, k, v, **kw)
    first = bcl.attention_bwd(q, k, v, o, lse, do, **kw)
    for _ in range(5):
        o2, lse2 = bcl.attention_fwd(q, k, v, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(first, bcl.attention_bwd(q, k, v, o, lse, do, **kw)):
            assert torch.equal(a, b)


def test_attention_workspace_given():
    x, kw, _, _ = au.case((13,), 1, 2, 900, 4, 2, 64, "f16")
    q, k, v, do = (x[n][0] for n in ("q", "k", "v", "dout"))
    o, lse = bcl.attention_fwd(q, k, v, **kw)
    ws = torch.full((1 << 22,), float("nan"), device=DEV)
    o2, lse2 = bcl.attention_fwd(q, k, v, ws=ws, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for a, b in zip(bcl.attention_bwd(q, k, v, o, lse, do, ws=ws, **kw)[:3], bcl.attention_bwd(q, k, v, o, lse, do, **kw)):
        assert torch.equal(a, b)
    with pytest.raises(bcl.FinetuneError):
        bcl.attention_bwd(q, k, v, o, lse, do, ws=ws[:4], **kw)


def test_calls_on_another_stream_and_in_a_graph():
    """The three operators captured together; replays between other work give the eager results on new inputs."""
    shape = (2, 130, 140, 4, 2, 64)
    x, kw, _, _ = au.case((14,), *shape, "bf16", table=16, spanned=True)
    q, k, v, do = (x[n][0].clone() for n in ("q", "k", "v", "dout"))
    seed = torch.tensor([5], device=DEV)

    def step(seed):
        o, lse = bcl.attention_fwd(q, k, v, **kw)
        y = bcl.dropout_fwd(o, 0.2, seed, 3, residual=do)
        dx = bcl.dropout_bwd(do, 0.2, seed, 3)
        grads = bcl.attention_bwd(q, k, v, o, lse, dx, **kw)
        bias = bcl.relative_bias_fwd(kw["bias"], 130, 140, kw["max_distance"])
        return [o, lse, y, dx, *grads, bias, bcl.relative_bias_bwd(bias, 16, kw["max_distance"])]

    want = step(seed)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(seed)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(bcl.dropout_bwd(do, 0.2, 5, 3, stream=side), want[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(seed)
    for n in range(4):
        q.copy_(torch.randn(q.shape, device=DEV))
        seed.fill_(100 + n)
        want = [t.clone() for t in step(100 + n)]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# relative position bias as a tensor
# ---------------------------------------------------------------------------
BIASES = [(1, 1, 1, 1), (2, 3, 5, 9), (1, 2, 40, 33), (3, 2, 300, 270), (1, 1, 1, 2500), (2, 1, 2100, 3), (1, 5, 257, 255)]
RULES = [(8, 20, True), (7, 20, False), (32, 128, True), (512, 1024, True), (2, 2, False), (4, 1024, True)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("shape", BIASES)
def test_relative_bias(shape, rule, dtype):
    b, h, tq, tk = shape
    count, distance, both = rule
    r = rng(20, *shape, count)
    table, ref = stored(r.standard_normal((count, h)), "f32")
    how = dict(max_distance=distance, bidirectional=both)
    got = bcl.relative_bias_fwd(table.to(DEV), tq, tk, dtype=TORCH[dtype], **how)
    want = torch.from_numpy(ao.relative_bias(ref, tq, tk, distance, both)).to(TORCH[dtype])
    assert torch.equal(got.cpu(), want)
    d, dr = stored(r.standard_normal((b, h, tq, tk)), dtype)
    total = ao.relative_bias_bwd(dr, count, distance, both)
    mag = ao.relative_bias_bwd(np.abs(dr), count, distance, both)
    # fp32 sums along a position's diagonal over the batch, then fp64
    within(f64(bcl.relative_bias_bwd(d.to(DEV), count, **how)), total, (b * tq + 8) * U * mag)


def test_relative_bias_strides():
    r = rng(21)
    wide = torch.from_numpy(r.standard_normal((2, 40, 3, 60))).to(DEV, torch.bfloat16)
    d = wide.transpose(1, 2)[..., 5:50]
    how = dict(max_distance=20)
    want = bcl.relative_bias_bwd(d.contiguous(), 8, **how)
    assert torch.equal(bcl.relative_bias_bwd(d, 8, **how), want)
    one = bcl.relative_bias_bwd(d[0], 8, **how)
    both = bcl.relative_bias_bwd(d[:1].expand(4, -1, -1, -1), 8, **how)
    within(f64(both), 4 * f64(one), 200 * U * f64(bcl.relative_bias_bwd(d[:1].abs(), 8, **how)) * 4)
    table = torch.full((8, 3), float("nan"), device=DEV)
    assert bcl.relative_bias_bwd(d, 8, dtable=table, **how) is table and torch.equal(table, want)
    assert not bcl.relative_bias_bwd(d[:, :, :0], 8, **how).any() and not bcl.relative_bias_bwd(d[:0], 8, **how).any()
    assert bcl.relative_bias_fwd(table, 0, 5, **how).shape == (3, 0, 5)


def test_bias_inside_and_outside_agree():
    """Gradients of the fused table, and of the bias as a tensor from ds of the whole matrix."""
    x, kw, see, bias = au.case((22,), 2, 150, 130, 2, 2, 32, "f32", table=8)
    q, k, v, do = (x[n][0] for n in ("q", "k", "v", "dout"))
    o, lse = bcl.attention_fwd(q, k, v, **kw)
    dbias = bcl.attention_bwd(q, k, v, o, lse, do, **kw)[3]
    _, _, p = ao.attention(*(x[n][1] for n in "qkv"), kw["scale"], see, bias)
    ds = ao.attention_bwd(*(x[n][1] for n in "qkv"), p, x["dout"][1], kw["scale"])[3]
    ds = torch.from_numpy(ds).to(DEV, torch.float32)
    apart = bcl.relative_bias_bwd(ds, 8, kw["max_distance"])
    assert (dbias - apart).norm() <= 1e-5 * apart.norm()


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
DROPS = [(1, 1), (1, 7), (1, 8), (3, 5), (5, 64), (1, 4096), (37, 1023), (300, 512)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", DROPS)
def test_dropout(shape, dtype):
    r = rng(30, *shape)
    (x, xr), (res, rr) = (stored(r.standard_normal(shape), dtype) for _ in range(2))
    x, res = x.to(DEV), res.to(DEV)
    for p, seed, offset in ((0.1, 7, 0), (0.5, (1 << 64) - 1, 1 << 40), (0.0, 3, 1), (1.0, 3, 1), (1e-7, 1, 2)):
        want = ao.dropout(xr, p, seed, offset)
        y = f64(bcl.dropout_fwd(x, p, seed, offset))
        within(y, want, store_err(want, dtype) + 4 * U * np.abs(want))
        assert np.array_equal(y == 0, want == 0)
        assert torch.equal(bcl.dropout_bwd(x, p, seed, offset), bcl.dropout_fwd(x, p, seed, offset))
        both = ao.dropout(xr, p, seed, offset, rr)
        got = f64(bcl.dropout_fwd(x, p, seed, offset, residual=res))
        within(got, both, store_err(both, dtype) + 4 * U * (np.abs(want) + np.abs(rr)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,gap", [((9, 8), 1), ((33, 21), 3), ((5, 1000), 8), ((64, 1), 6), ((20, 3), 2)])
def test_dropout_rows_apart(shape, gap, dtype):
    """The mask goes by the element's index, wherever its row stands; gaps are left alone."""
    r = rng(31, *shape, gap)
    wide = [stored(r.standard_normal((shape[0], shape[1] + gap)), dtype)[0].to(DEV) for _ in range(3)]
    x, res, y = (w[:, : shape[1]] for w in wide)
    rest = wide[2][:, shape[1]:].clone()
    want = bcl.dropout_fwd(x.contiguous(), 0.3, 11, 4, residual=res.contiguous())
    assert torch.equal(bcl.dropout_fwd(x, 0.3, 11, 4, residual=res), want)
    assert bcl.dropout_fwd(x, 0.3, 11, 4, residual=res, y=y) is y and torch.equal(y, want)
    assert torch.equal(wide[2][:, shape[1]:], rest)
    grad = bcl.dropout_bwd(x.contiguous(), 0.3, 11, 4)
    assert torch.equal(bcl.dropout_bwd(x, 0.3, 11, 4, dx=x), grad) and torch.equal(x, grad)


def test_dropout_in_place_and_offset_memory():
    r = rng(32)
    for dtype in DTYPES:
        base = stored(r.standard_normal(5003), dtype)[0].to(DEV)
        for start in (0, 1, 3):
            x = base[start:].clone()
            odd = torch.empty_like(base)[start:]  # starts off a piece's alignment
            odd.copy_(x)
            want = bcl.dropout_fwd(x, 0.2, 9)
            assert torch.equal(bcl.dropout_fwd(odd, 0.2, 9), want)
            assert torch.equal(bcl.dropout_fwd(odd, 0.2, 9, y=odd), want) and torch.equal(odd, want)
            both = bcl.dropout_fwd(x, 0.2, 9, residual=want)
            res = want.clone()
            assert torch.equal(bcl.dropout_fwd(x, 0.2, 9, residual=res, y=res), both)


def test_dropped_places_hide_what_they_held():
    x = torch.full((1000,), float("nan"), device=DEV)
    keep, _ = ao.dropout_keep(1000, 0.5, 4, 0)
    y = f64(bcl.dropout_fwd(x, 0.5, 4))
    assert np.array_equal(np.isnan(y), keep) and not y[~keep].any()


def test_dropout_seed_tensor():
    x = torch.randn(100, 40, device=DEV)
    for seed in (3, (1 << 63) - 1, -5):
        t = torch.tensor([seed], device=DEV)
        assert torch.equal(bcl.dropout_fwd(x, 0.4, t, 2), bcl.dropout_fwd(x, 0.4, seed % (1 << 64), 2))


def test_dropout_large():
    """More groups than one round of the launch's threads; past the caches."""
    x = torch.ones(1 << 15, 3000, device=DEV, dtype=torch.bfloat16)
    for n in (x.flatten()[: (1 << 22) + 5], x.flatten()):
        y = bcl.dropout_fwd(n, 0.25, 6, 1)
        least = round(0.25 * 65536)
        share = float((y == 0).float().mean())
        assert abs(share - least / 65536) < 6 * (0.25 * 0.75 / len(n)) ** 0.5
        keep, _ = ao.dropout_keep(len(n), 0.25, 6, 1)
        assert np.array_equal((y != 0).cpu().numpy(), keep)
        scale = torch.tensor(65536 / (65536 - least), device=DEV)
        want = torch.where(y == 0, torch.ones((), device=DEV), scale + 1).to(n.dtype)  # rounded once
        assert torch.equal(bcl.dropout_fwd(n, 0.25, 6, 1, residual=n), want)
