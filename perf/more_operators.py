"""Measured cases of a transformer sublayer's operators beside the circulant layers.

Three operators of a training step that store nothing of the size of the score
matrix or of a mask: attention whose backward recomputes the probabilities
(with a learned relative position bias fused in), that bias by itself with its
gradient, and dropout from a counter-based generator (with the residual sum).

``run`` computes a case with the package's operators where ``own`` is true and
otherwise in plain torch operations; ``exact`` computes it in 64 bits.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
MAX_FLOPS = 6.9e11  # of the largest listed case


def listed():
    return [
        # one new token after 4096 others in the D = 4096 layer's heads, four query heads to a key head: few rows,
        # a long axis
        dict(name="attn_fwd_token", op="attn", step="fwd", b=1, tq=1, tk=4096, hq=32, hk=8, d=128, dtype="bf16",
             causal=True, spans=False, bias=0),
        # the 2048 tokens of the adapter workload as four sequences
        dict(name="attn_fwd_tokens", op="attn", step="fwd", b=4, tq=512, tk=512, hq=32, hk=32, d=128, dtype="f16",
             causal=True, spans=False, bias=0),
        # odd lengths and an odd head size, a padded batch with an empty sequence, queries apart from the keys
        dict(name="attn_fwd_odd", op="attn", step="fwd", b=5, tq=333, tk=509, hq=12, hk=4, d=72, dtype="bf16",
             causal=False, spans=True, bias=0),
        # the D = 64 layer in 32 bits, four heads: latency of a backward call
        dict(name="attn_bwd_small", op="attn", step="bwd", b=2, tq=64, tk=64, hq=4, hk=2, d=16, dtype="f32",
             causal=True, spans=False, bias=0),
        # an encoder's padded batch with a position bias: its table's gradient from inside the attention
        dict(name="attn_bwd_bias", op="attn", step="bwd", b=8, tq=512, tk=512, hq=16, hk=16, d=64, dtype="bf16",
             causal=False, spans=True, bias=32),
        # long sequences, shared key heads
        dict(name="attn_bwd_long", op="attn", step="bwd", b=2, tq=4096, tk=4096, hq=32, hk=8, d=128, dtype="bf16",
             causal=True, spans=False, bias=0),
        # the bias of 16 heads over 512 positions, for an attention that takes it as a tensor
        dict(name="bias_fwd", op="bias", step="fwd", b=1, h=16, tq=512, tk=512, dtype="bf16", buckets=32,
             distance=128, both=True),
        # odd lengths in 32 bits, a decoder's one-sided buckets
        dict(name="bias_bwd_odd", op="bias", step="bwd", b=3, h=12, tq=1021, tk=1301, dtype="f32", buckets=31,
             distance=300, both=False),
        # the gradient from a batch of long sequences
        dict(name="bias_bwd_batch", op="bias", step="bwd", b=8, h=16, tq=2048, tk=2048, dtype="bf16", buckets=32,
             distance=128, both=True),
        # one token's activations: latency
        dict(name="drop_fwd_token", op="drop", step="fwd", rows=1, d=4096, dtype="bf16", p=0.1, residual=True,
             gap=0),
        # odd rows out of a wider buffer, backward in 32 bits
        dict(name="drop_bwd_odd", op="drop", step="bwd", rows=1021, d=1023, dtype="f32", p=0.3, residual=False,
             gap=5),
        # a long batch of the D = 4096 layer with the residual sum
        dict(name="drop_fwd_batch", op="drop", step="fwd", rows=16384, d=4096, dtype="bf16", p=0.1, residual=True,
             gap=0),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "bias", "drop"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    wide = 2 if dtype == "f32" else 1
    if op == "drop":
        d = _log(rng, 8, 16384)
        rows = _log(rng, 1, max(1, min(65536, (1 << 26) // wide // d)))
        return dict(op=op, step=rng.choice(["fwd", "bwd"]), rows=rows, d=d, dtype=dtype,
                    p=rng.choice([0.05, 0.1, 0.3, 0.5]), residual=rng.random() < 0.5,
                    gap=rng.choice([0, 0, 0, 8, 37]))
    if op == "bias":
        step = rng.choice(["fwd", "bwd"])
        b = _log(rng, 1, 8) if step == "bwd" else 1
        h, tq = _log(rng, 1, 32), _log(rng, 1, 2048)
        tk = _log(rng, 1, max(1, min(2048, (1 << 29) // wide // (b * h * tq))))
        both = rng.random() < 0.5
        return dict(op=op, step=step, b=b, h=h, tq=tq, tk=tk, dtype=dtype,
                    buckets=rng.choice([8, 32, 64]) if both else rng.choice([7, 32, 45]),
                    distance=rng.choice([64, 128, 500]), both=both)
    step = rng.choice(["fwd", "bwd"])
    d = rng.choice([16, 32, 64, 64, 80, 96, 128, 128, rng.randint(8, 127)])
    hk = _log(rng, 1, 16)
    hq = hk * rng.choice([1, 1, 2, 4])
    b = _log(rng, 1, 8)
    per = (4 if step == "fwd" else 10) * d * b * hq * (8 if dtype == "f32" else 1)  # 32 bits run at an eighth or less
    pairs = min(MAX_FLOPS / per, 5e8 / (b * hq))
    shape = rng.choice(["square", "square", "cross", "few"])
    if shape == "square":
        tq = tk = _log(rng, 1, max(1, min(4096, int(math.sqrt(pairs)))))
    elif shape == "few":  # few queries on a long axis
        tq = _log(rng, 1, 16)
        tk = _log(rng, 64, max(64, min(16384, int(pairs / tq))))
    else:
        tq = _log(rng, 1, max(1, min(2048, int(math.sqrt(pairs)))))
        tk = _log(rng, 1, max(1, min(4096, int(pairs / tq))))
    return dict(op=op, step=step, b=b, tq=tq, tk=tk, hq=hq, hk=hk, d=d, dtype=dtype, causal=rng.random() < 0.6,
                spans=rng.random() < 0.4, bias=rng.choice([0, 0, 32]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
ATTN_DISTANCE = 128  # max_distance of the bias inside the attention; its buckets are one-sided where it is causal


def _spans(b, t):
    """[begin, end) of the keys that count in each of b sequences of t
    positions: padding on either side, the last of four or more all padding;
    fixed by b and t alone."""
    r = random.Random(1000003 * b + t)
    out = []
    for i in range(b):
        lo = int(r.uniform(0.0, 0.3) * t) if r.random() < 0.5 else 0
        hi = t - int(r.uniform(0.0, 0.5) * t)
        out.append((0, 0) if b >= 4 and i == b - 1 else (lo, max(hi, lo + 1)))
    return out


def _scale(case):
    return 1.0 / math.sqrt(case["d"])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).add_(mean).to(dtype)

    s = {"case": case}
    dt = DT[case["dtype"]]
    if case["op"] == "drop":
        rows, d = case["rows"], case["d"]
        s["x"] = normal(rows, d + case["gap"], dtype=dt)[:, :d]  # upstream gradient in a backward
        s["residual"] = normal(rows, d, dtype=dt) if case["residual"] and case["step"] == "fwd" else None
        s["seed"], s["offset"] = (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), seed % 1000
        return s
    if case["op"] == "bias":
        if case["step"] == "fwd":
            s["table"] = normal(case["buckets"], case["h"])
        else:
            s["dbias"] = normal(case["b"], case["h"], case["tq"], case["tk"], mean=0.02, dtype=dt)
        return s
    b, tq, tk, hq, hk, d = (case[k] for k in ("b", "tq", "tk", "hq", "hk", "d"))
    if tq == tk:  # as a fused projection leaves them: views of one buffer
        qkv = normal(b, tq, hq + 2 * hk, d, scale=1.3, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
    else:
        s["q"] = normal(b, tq, hq, d, scale=1.3, dtype=dt)
        kv = normal(2, b, tk, hk, d, scale=1.3, dtype=dt)
        s["k"], s["v"] = kv[0], kv[1]
    s["begin"] = s["end"] = None
    if case["spans"]:
        spans = torch.tensor(_spans(b, tk), device=DEV, dtype=torch.int32)
        s["begin"], s["end"] = spans[:, 0].contiguous(), spans[:, 1].contiguous()
    s["table"] = normal(case["bias"], hq, scale=0.5) if case["bias"] else None
    if case["step"] == "bwd":  # what the forward pass left behind, and the upstream gradient
        s["dout"] = normal(b, tq, hq, d, dtype=dt)
        s["o"] = torch.empty(b, tq, hq, d, device=DEV, dtype=dt)
        s["lse"] = torch.empty(b, hq, tq, device=DEV)
        for i in range(b):
            for n in range(hk):
                heads = slice(n * (hq // hk), (n + 1) * (hq // hk))
                o, lse, _ = _attend64(s, i, n)
                s["o"][i, :, heads] = o.transpose(0, 1).to(dt)
                s["lse"][i, heads] = lse.float()
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import block_circulant_layers_amd as bcl

    case = s["case"]
    if case["op"] == "drop":
        if case["step"] == "fwd":
            return {"y": bcl.dropout_fwd(s["x"], case["p"], s["seed"], s["offset"], residual=s["residual"])}
        return {"dx": bcl.dropout_bwd(s["x"], case["p"], s["seed"], s["offset"])}
    if case["op"] == "bias":
        how = dict(max_distance=case["distance"], bidirectional=case["both"])
        if case["step"] == "fwd":
            return {"bias": bcl.relative_bias_fwd(s["table"], case["tq"], case["tk"], dtype=DT[case["dtype"]], **how)}
        return {"dtable": bcl.relative_bias_bwd(s["dbias"], case["buckets"], **how)}
    how = dict(scale=_scale(case), causal=case["causal"], key_begin=s["begin"], key_end=s["end"], bias=s["table"],
               max_distance=ATTN_DISTANCE, bidirectional=not case["causal"])
    if case["step"] == "fwd":
        o, lse = bcl.attention_fwd(s["q"], s["k"], s["v"], **how)
        return {"o": o, "lse": lse}
    dq, dk, dv, dbias = bcl.attention_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], **how)
    return {"dq": dq, "dk": dk, "dv": dv, "dbias": dbias}


def _run_plain(s):
    """The operators in elementary operations, rounded to the storage type at the end."""
    case = s["case"]
    return {"attn": _attn, "bias": _bias, "drop": _drop}[case["op"]](s, case)


def _bucket(rel, buckets, distance, both):
    """The bucket of each relative position rel = key - query (in 64 bits: the
    logarithm's borders are met exactly)."""
    if both:
        buckets //= 2
        base, n = torch.where(rel > 0, buckets, 0), rel.abs()
    else:
        base, n = torch.zeros_like(rel), (-rel).clamp(min=0)
    small = buckets // 2
    far = (n.clamp(min=1).double() / small).log() / math.log(distance / small) * (buckets - small)
    far = (small + (far + 1e-9).floor().long()).clamp(max=buckets - 1)
    return base + torch.where(n < small, n, far)


def _positions(tq, tk):
    """key - query of every pair; the last query stands at the last key."""
    return torch.arange(tk, device=DEV) - (torch.arange(tq, device=DEV)[:, None] + (tk - tq))


def _by_bucket(x, bucket, buckets):
    """x (heads, queries, keys) summed by bucket: along diagonals first (the
    rows, last one first, each shifted by one), then 64-bit sums."""
    h, tq, tk = x.shape
    w = tq + tk - 1
    skew = torch.nn.functional.pad(x.flip(1), (0, tq)).reshape(h, -1)[:, :tq * w].view(h, tq, w)
    along = skew.sum(1, dtype=torch.float64)  # column m: key - query = m - (tq - 1) before the shift to the last key
    return torch.zeros(buckets, h, device=DEV, dtype=torch.float64).index_add_(0, bucket, along.t()).float()


def _diagonals(tq, tk, buckets, distance, both):
    return _bucket(torch.arange(tq + tk - 1, device=DEV) - (tk - 1), buckets, distance, both)


def _bias(s, case):
    how = (case["buckets"], case["distance"], case["both"])
    tq, tk = case["tq"], case["tk"]
    if case["step"] == "fwd":
        return {"bias": s["table"][_bucket(_positions(tq, tk), *how)].permute(2, 0, 1).to(DT[case["dtype"]]).contiguous()}
    return {"dtable": _by_bucket(s["dbias"].sum(0, dtype=torch.float32), _diagonals(tq, tk, *how), case["buckets"])}


def _attn(s, case):
    b, tq, tk, hq, hk, d = (case[k] for k in ("b", "tq", "tk", "hq", "hk", "d"))
    group, dt = hq // hk, DT[case["dtype"]]
    how = (case["bias"], ATTN_DISTANCE, not case["causal"])

    def rows(t):  # (b, key heads, query heads of a key head * tq, d)
        return t.float().permute(0, 2, 1, 3).reshape(b, hk, group * tq, d)

    def back(t):
        return t.view(b, hq, tq, d).permute(0, 2, 1, 3).to(dt).contiguous()

    q, k, v = rows(s["q"]), s["k"].float().permute(0, 2, 1, 3), s["v"].float().permute(0, 2, 1, 3)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(_scale(case)).view(b, hq, tq, tk)
    rel = _positions(tq, tk)
    if case["bias"]:
        x += s["table"][_bucket(rel, *how)].permute(2, 0, 1)
    hidden = torch.zeros(1, 1, tq, tk, device=DEV, dtype=torch.bool)
    if case["causal"]:
        hidden = hidden | (rel > 0)
    if case["spans"]:
        j = torch.arange(tk, device=DEV)
        hidden = hidden | ((j < s["begin"][:, None]) | (j >= s["end"][:, None]))[:, None, None]
    if case["causal"] or case["spans"]:
        x.masked_fill_(hidden, -math.inf)
    if case["step"] == "fwd":
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        lse = (top + total.log())[..., 0]
        o = torch.matmul(p.view(b, hk, group * tq, tk), v).view(b, hq, tq, d) / torch.where(total == 0, 1.0, total)
        return {"o": back(o), "lse": lse}
    lse = s["lse"][..., None]
    p = x.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_().view(b, hk, group * tq, tk)
    dout = rows(s["dout"])
    dp = torch.matmul(dout, v.transpose(2, 3))
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p)
    out = {"dq": back(torch.matmul(ds, k) * _scale(case)),
           "dk": (torch.matmul(ds.transpose(2, 3), q) * _scale(case)).permute(0, 2, 1, 3).to(dt).contiguous(),
           "dv": torch.matmul(p.transpose(2, 3), dout).permute(0, 2, 1, 3).to(dt).contiguous(), "dbias": None}
    if case["bias"]:
        out["dbias"] = _by_bucket(ds.view(b, hq, tq, tk).sum(0), _diagonals(tq, tk, *how), case["bias"])
    return out


_MUL, _ADD = (0xD2511F53, 0xCD9E8D57), (0x9E3779B9, 0xBB67AE85)  # of Philox4x32 (Salmon et al., SC 2011)
_LOW = 0xFFFFFFFF


def _words(blocks, seed, offset):
    """Philox4x32-10 of the counters (block, offset) under the key seed: four 32-bit words a block."""
    n = torch.arange(blocks, device=DEV)
    c0, c1 = n & _LOW, n >> 32
    c2, c3 = torch.full_like(n, offset & _LOW), torch.full_like(n, offset >> 32)
    k0, k1 = seed & _LOW, seed >> 32
    for _ in range(10):
        a, c = c0 * _MUL[0], c2 * _MUL[1]
        c0, c1, c2, c3 = ((c >> 32) & _LOW) ^ c1 ^ k0, c & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = (k0 + _ADD[0]) & _LOW, (k1 + _ADD[1]) & _LOW
    return torch.stack([c0, c1, c2, c3], -1)


def _drop(s, case):
    rows, d = case["rows"], case["d"]
    words = _words(-(-rows * d // 8), s["seed"], s["offset"])
    bits = torch.stack([words & 0xFFFF, words >> 16], -1).view(-1)[:rows * d].view(rows, d)
    least = round(case["p"] * 65536)  # an element is dropped where its 16 bits are below
    y = torch.where(bits >= least, s["x"].float() * (65536 / (65536 - least)), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y" if case["step"] == "fwd" else "dx": y.to(DT[case["dtype"]])}


# ---------------------------------------------------------------------------
# floors and the 64-bit values
# ---------------------------------------------------------------------------
def work(case):
    """Bytes that have to move and operations that have to be done once."""
    e = SIZE[case["dtype"]]
    if case["op"] == "drop":
        n = case["rows"] * case["d"]
        reads = 2 if case["residual"] and case["step"] == "fwd" else 1
        # ten rounds of two products and six other operations for eight elements, and four for each
        return {"bytes": (reads + 1) * n * e, "flops": 14 * n}
    if case["op"] == "bias":
        n = case["h"] * case["tq"] * case["tk"]
        return {"bytes": case["b"] * n * e + case["buckets"] * case["h"] * 4, "flops": case["b"] * n}
    b, tq, tk, hq, hk, d = (case[k] for k in ("b", "tq", "tk", "hq", "hk", "d"))
    spans = _spans(b, tk) if case["spans"] else [(0, tk)] * b
    keys = sum(hi - lo for lo, hi in spans)
    pairs = sum(max(0, min(hi, i + tk - tq + 1) - lo) if case["causal"] else hi - lo
                for lo, hi in spans for i in range(tq))
    small = b * hq * tq * 4 + case["bias"] * hq * 4
    if case["step"] == "fwd":
        return {"bytes": (2 * b * tq * hq + 2 * keys * hk) * d * e + small, "flops": 4 * pairs * hq * d}
    return {"bytes": (4 * b * tq * hq + 2 * (keys + b * tk) * hk) * d * e + small, "flops": 10 * pairs * hq * d}


def _buckets_of(reach, buckets, distance, both):
    """bucket(rel) for |rel| <= reach by whole-number comparisons: bucket small + m
    begins at the first n with (n / small)^rest >= (distance / small)^m."""
    half = buckets // 2 if both else buckets
    small = half // 2
    rest, one, m = half - small, [], 0
    for n in range(reach + 1):
        if n >= small:
            while m + 1 < rest and n**rest * small**(m + 1) >= distance**(m + 1) * small**rest:
                m += 1
        one.append(n if n < small else small + m)
    later = [half + x for x in one] if both else [0] * (reach + 1)
    return torch.tensor(one[:0:-1] + [one[0]] + later[1:], device=DEV)


def _bucket_table(case_buckets, tq, tk, distance, both):
    i, j = torch.arange(tq, device=DEV) + (tk - tq), torch.arange(tk, device=DEV)
    reach = tq + tk
    return _buckets_of(reach, case_buckets, distance, both)[j[None, :] - i[:, None] + reach]


def _attend64(s, i, n, leaves=False):
    """Sequence i, key head n in 64 bits: (o, lse, leaves), heads first."""
    case = s["case"]
    tq, tk, group = case["tq"], case["tk"], case["hq"] // case["hk"]
    heads = slice(n * group, (n + 1) * group)
    q, k, v = s["q"][i, :, heads].double().transpose(0, 1), s["k"][i, :, n].double(), s["v"][i, :, n].double()
    x0 = torch.zeros(group, tq, tk, device=DEV, dtype=torch.float64)
    if case["bias"]:
        where = _bucket_table(case["bias"], tq, tk, ATTN_DISTANCE, not case["causal"])
        x0 = torch.stack([s["table"][:, h].double()[where] for h in range(n * group, (n + 1) * group)])
    if leaves:
        q, k, v, x0 = (t.clone().requires_grad_(True) for t in (q, k, v, x0))
    j = torch.arange(tk, device=DEV)
    seen = torch.ones(tq, tk, device=DEV, dtype=torch.bool)
    if case["causal"]:
        seen = j <= torch.arange(tq, device=DEV)[:, None] + (tk - tq)
    if case["spans"]:
        seen = seen & (j >= s["begin"][i]) & (j < s["end"][i])
    x = torch.einsum("gqd,kd->gqk", q, k) * _scale(case) + x0
    live = seen.any(-1)
    x = torch.where(seen | ~live[:, None], x, -math.inf)
    p = torch.softmax(x, -1) * live[:, None]
    lse = torch.where(live, torch.logsumexp(x.detach(), -1), -math.inf)
    return torch.einsum("gqk,kd->gqd", p, v), lse, (q, k, v, x0)


def exact(case, seed):
    """The definitions in float64; the attention's gradients by autograd."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "drop":
        rows, d = case["rows"], case["d"]
        c = np.arange(-(-rows * d // 8), dtype=np.uint64)
        c = [c & np.uint64(_LOW), c >> np.uint64(32), np.full_like(c, s["offset"] & _LOW),
             np.full_like(c, s["offset"] >> 32)]
        key = [s["seed"] & _LOW, s["seed"] >> 32]
        for r in range(10):
            x, y = c[0] * np.uint64(_MUL[0]), c[2] * np.uint64(_MUL[1])
            k = [np.uint64((a + r * w) & _LOW) for a, w in zip(key, _ADD)]
            c = [(y >> np.uint64(32)) ^ c[1] ^ k[0], y & np.uint64(_LOW), (x >> np.uint64(32)) ^ c[3] ^ k[1],
                 x & np.uint64(_LOW)]
        half = np.stack(c, -1).astype(np.uint32).view(np.uint16).reshape(-1)[:rows * d]
        least = round(case["p"] * 65536)
        keep = torch.from_numpy((half >= least).reshape(rows, d)).to(DEV)
        y = s["x"].to(f) * keep / (1 - least / 65536)
        if s["residual"] is not None:
            y = y + s["residual"].to(f)
        return {"y" if case["step"] == "fwd" else "dx": y}
    if case["op"] == "bias":
        where = _bucket_table(case["buckets"], case["tq"], case["tk"], case["distance"], case["both"])
        if case["step"] == "fwd":
            return {"bias": torch.stack([col[where] for col in s["table"].to(f).t()])}
        total = torch.zeros(case["h"], case["buckets"], device=DEV, dtype=f)
        for one in s["dbias"]:
            total.index_add_(1, where.flatten(), one.to(f).flatten(1))
        return {"dtable": total.t()}
    b, tq, tk, hq, hk, d = (case[k] for k in ("b", "tq", "tk", "hq", "hk", "d"))
    group = hq // hk
    if case["step"] == "fwd":
        o, lse = torch.empty(b, tq, hq, d, device=DEV, dtype=f), torch.empty(b, hq, tq, device=DEV, dtype=f)
        for i in range(b):
            for n in range(hk):
                heads = slice(n * group, (n + 1) * group)
                one, lse[i, heads], _ = _attend64(s, i, n)
                o[i, :, heads] = one.transpose(0, 1)
        return {"o": o, "lse": lse}
    dq = torch.empty(b, tq, hq, d, device=DEV, dtype=f)
    dk, dv = torch.empty(b, tk, hk, d, device=DEV, dtype=f), torch.empty(b, tk, hk, d, device=DEV, dtype=f)
    table = torch.zeros(hq, max(case["bias"], 1), device=DEV, dtype=f)
    where = _bucket_table(case["bias"], tq, tk, ATTN_DISTANCE, not case["causal"]) if case["bias"] else None
    for i in range(b):
        for n in range(hk):
            heads = slice(n * group, (n + 1) * group)
            o, _, leaves = _attend64(s, i, n, leaves=True)
            gq, gk, gv, gx = torch.autograd.grad(o, leaves, s["dout"][i, :, heads].to(f).transpose(0, 1))
            dq[i, :, heads], dk[i, :, n], dv[i, :, n] = gq.transpose(0, 1), gk, gv
            if case["bias"]:
                table[heads].index_add_(1, where.flatten(), gx.flatten(1))
    return {"dq": dq, "dk": dk, "dv": dv, "dbias": table.t() if case["bias"] else None}
