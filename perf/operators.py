"""Measured cases of the fine-tuning operators beside the circulant layers.

Four operators of a fine-tuning step: layer normalisation (forward and
backward), the pairwise preference loss and the clipped policy loss on
vocabulary logits (forward, and forward with the gradient of the logits), and
the global gradient norm with clipping over a list of tensors.

``run`` computes a case with the package's operators where ``own`` is true and
otherwise in plain 32-bit torch operations; ``exact`` computes it in 64 bits.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
IGNORE = -100  # label of a position that takes no part in a loss


def listed():
    return [
        # one token through a normalisation of the D = 4096 layer: latency alone
        dict(name="norm_fwd_token", op="norm", step="fwd", rows=1, d=4096, dtype="bf16", bias=True),
        # the 2048 tokens of the adapter workload, forward
        dict(name="norm_fwd_tokens", op="norm", step="fwd", rows=2048, d=4096, dtype="f16", bias=True),
        # odd row count and width in 32 bits, no bias: rows that start at any multiple of 4 bytes
        dict(name="norm_bwd_odd", op="norm", step="bwd", rows=1021, d=1023, dtype="f32", bias=False),
        # a long batch of the D = 4096 layer, backward: dx and the sums over tokens
        dict(name="norm_bwd_batch", op="norm", step="bwd", rows=16384, d=4096, dtype="bf16", bias=True),
        # one short pair and a small vocabulary: latency of a whole loss step
        dict(name="pref_step_pair", op="pref", step="step", pairs=1, t=16, v=1009, dtype="f32", kind="ipo",
             smoothing=0.0, average=True),
        # held-out pairs scored without a gradient
        dict(name="pref_eval", op="pref", step="fwd", pairs=8, t=512, v=32768, dtype="f16", kind="hinge",
             smoothing=0.0, average=False),
        # a training batch of pairs, odd vocabulary, prompts and padding masked
        dict(name="pref_step_batch", op="pref", step="step", pairs=4, t=1024, v=50001, dtype="bf16", kind="sigmoid",
             smoothing=0.1, average=False),
        # a few short answers over a wide vocabulary: fewer rows than compute units
        dict(name="policy_step_short", op="policy", step="step", seqs=4, t=8, v=32768, dtype="f16", ref=False,
             reduction="sequence"),
        # loss values only, odd sizes in 32 bits
        dict(name="policy_fwd_odd", op="policy", step="fwd", seqs=3, t=333, v=10007, dtype="f32", ref=True,
             reduction="token"),
        # a training batch over a large vocabulary
        dict(name="policy_step_batch", op="policy", step="step", seqs=8, t=1024, v=131072, dtype="bf16", ref=True,
             reduction="token"),
        # the gradients of 128 adapter layers 4096 x 4096 at p = 1024 (16384 floats each)
        dict(name="clip_adapters", op="clip", tensors=128, elems=128 * 16384, dtype="f32", spread=0.0, max_norm=1.0),
        # a whole model's gradients: uneven tensors of 32 and 16 bits
        dict(name="clip_model", op="clip", tensors=200, elems=1 << 28, dtype="mixed", spread=6.0, max_norm=1.0),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["norm", "pref", "policy", "clip"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    room = 2 if dtype == "f32" else 1  # a 32-bit case costs no more than the largest 16-bit one
    if op == "norm":
        d = _log(rng, 8, 16384)
        rows = _log(rng, 1, max(1, min(65536, 16384 * 4096 // room // d)))
        return dict(op=op, step=rng.choice(["fwd", "bwd"]), rows=rows, d=d, dtype=dtype, bias=rng.random() < 0.6)
    if op == "clip":
        dtype = rng.choice([dtype, "mixed"])
        tensors = _log(rng, 1, 400)
        return dict(op=op, tensors=tensors, elems=_log(rng, max(tensors, 1000), 1 << 27), dtype=dtype,
                    spread=rng.choice([0.0, 3.0, 6.0]), max_norm=rng.choice([0.5, 1.0, 1e9]))
    v = _log(rng, 16, 131072)
    rows = _log(rng, 2, max(2, min(16384, 8192 * 50001 // room // v)))
    if op == "pref":
        pairs = _log(rng, 1, max(1, min(16, rows // 2)))
        return dict(op=op, step=rng.choice(["fwd", "step"]), pairs=pairs, t=max(1, rows // (2 * pairs)), v=v,
                    dtype=dtype, kind=rng.choice(["sigmoid", "hinge", "ipo"]), smoothing=rng.choice([0.0, 0.1]),
                    average=rng.random() < 0.5)
    seqs = _log(rng, 1, min(32, rows))
    return dict(op=op, step=rng.choice(["fwd", "step"]), seqs=seqs, t=max(1, rows // seqs), v=v, dtype=dtype,
                ref=rng.random() < 0.7, reduction=rng.choice(["token", "sequence"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _spans(n, t):
    """[begin, end) of the answer in each of n sequences of t positions: a
    prompt before it, padding after it; fixed by n and t alone."""
    r = random.Random(1000003 * n + t)
    out = []
    for _ in range(n):
        b = int(r.uniform(0.0, 0.4) * t)
        e = t - int(r.uniform(0.0, 0.3) * t)
        out.append((b, max(e, b + 1)))
    return out


def _valid(n, t):
    return sum(e - b for b, e in _spans(n, t))


def _sizes(case):
    """Element counts of the tensors of a clip case, near case["elems"] in all."""
    r = random.Random(7919 * case["tensors"] + case["elems"])
    w = [math.exp(r.uniform(0.0, case["spread"])) for _ in range(case["tensors"])]
    return [max(1, int(case["elems"] * x / sum(w))) for x in w]


def _kinds(case):
    one = case["dtype"]
    return ["f32" if i % 2 else "bf16" for i in range(case["tensors"])] if one == "mixed" else [one] * case["tensors"]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).add_(mean).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op == "norm":
        rows, d, dt = case["rows"], case["d"], DT[case["dtype"]]
        s["x"] = normal(rows, d, scale=1.5, mean=0.3, dtype=dt)
        s["weight"] = normal(d, scale=0.2, mean=1.0)
        s["bias"] = normal(d, scale=0.2) if case["bias"] else None
        if case["step"] == "bwd":  # what the forward pass left behind
            s["dy"] = normal(rows, d, dtype=dt)
            x = s["x"].double()
            mean = x.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = (x - mean[:, None]).square().mean(-1).add(1e-5).rsqrt().float()
        return s
    if op == "clip":
        # as buckets of gradients hold them: the tensors of one type packed one after another, any element boundary
        sizes, kinds = _sizes(case), _kinds(case)
        total = {k: sum(n for n, kind in zip(sizes, kinds) if kind == k) for k in dict.fromkeys(kinds)}
        held = {k: normal(n, scale=1e-2, dtype=DT[k]) for k, n in total.items()}
        s["clipped"] = {k: torch.empty_like(t) for k, t in held.items()}
        s["grads"], s["out"], at = [], [], dict.fromkeys(held, 0)
        for n, k in zip(sizes, kinds):
            s["grads"].append(held[k][at[k]:at[k] + n])
            s["out"].append(s["clipped"][k][at[k]:at[k] + n])
            at[k] += n
        return s
    n = 2 * case["pairs"] if op == "pref" else case["seqs"]
    t, v = case["t"], case["v"]
    tokens = torch.randint(0, v, (n, t), generator=g, device=DEV)
    boost = torch.rand(n, t, 1, generator=g, device=DEV).mul_(10.0)
    logits = torch.randn(n, t, v, generator=g, device=DEV).mul_(2.0)
    logits.scatter_add_(2, tokens[..., None], boost)
    s["logits"] = logits = logits.to(DT[case["dtype"]])
    pos = torch.arange(t, device=DEV)
    span = torch.tensor(_spans(n, t), device=DEV)
    keep = (pos >= span[:, :1]) & (pos < span[:, 1:])
    s["labels"] = torch.where(keep, tokens, torch.full_like(tokens, IGNORE))
    logp = logits.gather(2, tokens[..., None])[..., 0].float() - torch.logsumexp(logits.float(), -1)
    if op == "pref":  # token log-probabilities of the frozen reference
        s["ref_logp"] = logp + normal(n, t, scale=0.2, mean=-0.01)
    else:  # ... and of the policy that sampled the answers; one advantage a sequence
        s["old_logp"] = logp + normal(n, t, scale=0.3)
        s["ref_logp"] = logp + normal(n, t, scale=0.3) if case["ref"] else None
        s["advantages"] = normal(n, 1)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
EPS = 1e-5
BETA = 0.1
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.05


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import block_circulant_layers_amd as bcl

    case = s["case"]
    if case["op"] == "norm":
        if case["step"] == "fwd":
            y, mean, rstd = bcl.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = bcl.layer_norm_bwd(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], need_db=case["bias"])
        return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}
    if case["op"] == "pref":
        how = dict(beta=BETA, kind=case["kind"], label_smoothing=case["smoothing"], average=case["average"])
        if case["step"] == "fwd":
            r = bcl.preference_loss_fwd(s["logits"], s["labels"], s["ref_logp"], **how)
            return {"loss": r.loss, "logratio": r.logratio, "logp": r.logp}
        r, dlogits = bcl.preference_loss_step(s["logits"], s["labels"], s["ref_logp"], scale=1.0 / case["pairs"],
                                              **how)
        return {"loss": r.loss, "logratio": r.logratio, "logp": r.logp, "dlogits": dlogits}
    if case["op"] == "policy":
        how = dict(ref_logp=s["ref_logp"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL,
                   reduction=case["reduction"])
        if case["step"] == "fwd":
            r = bcl.policy_loss_fwd(s["logits"], s["labels"], s["old_logp"], s["advantages"], **how)
            return {"loss": r.loss, "kl": r.kl, "logp": r.logp}
        r, dlogits = bcl.policy_loss_step(s["logits"], s["labels"], s["old_logp"], s["advantages"], scale=1.0, **how)
        return {"loss": r.loss, "kl": r.kl, "logp": r.logp, "dlogits": dlogits}
    norm = bcl.clip_grad_norm(s["grads"], case["max_norm"], out=s["out"])
    return {"norm": norm, **s["clipped"]}


def _run_plain(s):
    """The operators in elementary 32-bit operations, rounded to the storage type at the end."""
    case, wide = s["case"], torch.float32
    if case["op"] == "norm":
        return _norm_fwd(s, wide) if case["step"] == "fwd" else _norm_bwd(s, wide)
    if case["op"] == "clip":
        sums = torch.stack([g.to(wide).square().sum() for g in s["grads"]])
        norm = sums.sum().sqrt()
        scale = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        [o.copy_(g.to(wide).mul(scale)) for g, o in zip(s["grads"], s["out"])]
        return {"norm": norm, **s["clipped"]}
    x, labels = s["logits"].to(wide), s["labels"]
    keep = labels != IGNORE
    pick = labels.clamp(min=0)[..., None]
    top = x.amax(-1, keepdim=True)
    lse = top + (x - top).exp().sum(-1, keepdim=True).log()
    logp = torch.where(keep, (x.gather(2, pick) - lse)[..., 0], 0.0)
    out, per_token = (_pref if case["op"] == "pref" else _policy)(s, logp, keep, wide)
    out["logp"] = logp
    if case["step"] == "step":
        # d loss / d logits = g (onehot - softmax), g = d loss / d logp
        d = (x - lse).exp().neg()
        d.scatter_add_(2, pick, torch.ones_like(logp)[..., None])
        out["dlogits"] = torch.where(keep[..., None], d * per_token[..., None], 0.0).to(s["logits"].dtype)
    return out


def _pref(s, logp, keep, wide):
    case = s["case"]
    pairs, sm = case["pairs"], case["smoothing"]
    each = torch.where(keep, logp - s["ref_logp"].to(wide), 0.0)
    count = keep.sum(-1).to(wide).clamp(min=1.0) if case["average"] else torch.ones_like(each[:, 0])
    logratio = each.sum(-1) / count
    h = logratio[:pairs] - logratio[pairs:]
    z = BETA * h
    if case["kind"] == "sigmoid":
        log_up = torch.minimum(z, torch.zeros_like(z)) - torch.log1p((-z.abs()).exp())  # log sigmoid(z)
        loss = -(1 - sm) * log_up - sm * (log_up - z)
        slope = -BETA * ((1 - sm) / (1 + z.exp()) - sm / (1 + (-z).exp()))
    elif case["kind"] == "hinge":
        loss = (1 - z).clamp(min=0.0)
        slope = torch.where(z < 1, -BETA, 0.0).to(wide)
    else:
        loss = (h - 0.5 / BETA).square()
        slope = 2 * (h - 0.5 / BETA)
    per_seq = torch.cat([slope, -slope]) / count / pairs
    return {"loss": loss, "logratio": logratio}, per_seq[:, None] * keep


def _policy(s, logp, keep, wide):
    case = s["case"]
    ratio = torch.where(keep, logp - s["old_logp"].to(wide), 0.0).exp()
    adv = s["advantages"].to(wide).expand_as(logp)
    free, held = ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
    each, slope = -torch.minimum(free, held), torch.where(free <= held, -free, 0.0)
    kl = torch.zeros_like(logp)
    if s["ref_logp"] is not None:
        gap = torch.where(keep, s["ref_logp"].to(wide) - logp, 0.0)
        kl = torch.expm1(gap) - gap
        each, slope = each + KL * kl, slope - KL * torch.expm1(gap)
    if case["reduction"] == "token":
        w = keep / keep.sum().clamp(min=1).to(wide)
    else:
        w = keep / keep.sum(-1, keepdim=True).clamp(min=1).to(wide) / keep.shape[0]
    return {"loss": (each * w).sum(), "kl": (kl * w).sum()}, slope * w


def _norm_fwd(s, wide):
    x = s["x"].to(wide)
    mean = x.mean(-1, keepdim=True)
    mid = x - mean
    rstd = 1.0 / (mid.square().mean(-1, keepdim=True) + EPS).sqrt()
    y = mid * rstd * s["weight"].to(wide)
    if s["bias"] is not None:
        y = y + s["bias"].to(wide)
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _norm_bwd(s, wide):
    x, dy = s["x"].to(wide), s["dy"].to(wide)
    mean, rstd = s["mean"].to(wide)[:, None], s["rstd"].to(wide)[:, None]
    hat = (x - mean) * rstd
    g = dy * s["weight"].to(wide)
    dx = rstd * (g - g.mean(-1, keepdim=True) - hat * (g * hat).mean(-1, keepdim=True))
    out = {"dx": dx.to(s["x"].dtype), "dw": (dy * hat).sum(0)}
    if s["case"]["bias"]:
        out["db"] = dy.sum(0)
    return out


# ---------------------------------------------------------------------------
# floors and the 64-bit values
# ---------------------------------------------------------------------------
def work(case):
    """Bytes that have to move and operations that have to be done once."""
    op = case["op"]
    if op == "norm":
        n, e = case["rows"] * case["d"], SIZE[case["dtype"]]
        extra = case["rows"] * 8 + case["d"] * 4 * (2 if case["bias"] else 1)
        if case["step"] == "fwd":
            return {"bytes": 2 * n * e + extra, "flops": 8 * n}
        return {"bytes": 3 * n * e + extra + case["d"] * 4, "flops": 14 * n}
    if op == "clip":
        b = sum(n * SIZE[k] for n, k in zip(_sizes(case), _kinds(case)))
        return {"bytes": 2 * b, "flops": 3 * sum(_sizes(case))}
    n = 2 * case["pairs"] if op == "pref" else case["seqs"]
    e, v, t = SIZE[case["dtype"]], case["v"], case["t"]
    used = _valid(n, t)  # masked positions are not read; their gradient rows are written
    small = n * t * (8 + 4 + 4 + 4)
    if case["step"] == "fwd":
        return {"bytes": used * v * e + small, "flops": 4 * used * v}
    return {"bytes": used * v * e + n * t * v * e + small, "flops": 7 * used * v}


def exact(case, seed):
    """The definitions in float64: softmax, variance and norms written as such."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        x, w = s["x"].to(f), s["weight"].to(f)
        if case["step"] == "fwd":
            var, mean = torch.var_mean(x, dim=-1, correction=0)
            rstd = (var + EPS) ** -0.5
            y = torch.addcmul(s["bias"].to(f) if case["bias"] else torch.zeros_like(w), (x.T - mean).T * w,
                              rstd[:, None])
            return {"y": y, "mean": mean, "rstd": rstd}
        # dx = J^T (w dy) with J = rstd (I - 1 1^T / d - hat hat^T / d)
        hat = torch.einsum("rd,r->rd", x - s["mean"].to(f)[:, None], s["rstd"].to(f))
        dy = s["dy"].to(f)
        g = dy * w
        along = (g * hat).sum(-1, keepdim=True) / case["d"]
        flat = g.sum(-1, keepdim=True) / case["d"]
        out = {"dx": (g - flat - along * hat) * s["rstd"].to(f)[:, None], "dw": torch.einsum("rd,rd->d", dy, hat)}
        return {**out, "db": dy.sum(0)} if case["bias"] else out
    if case["op"] == "clip":
        norm = torch.sqrt(sum(torch.dot(g.to(f), g.to(f)) for g in s["grads"]))
        scale = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        flat = {k: torch.cat([g for g in s["grads"] if g.dtype == DT[k]]).to(f) * scale for k in s["clipped"]}
        return {"norm": norm, **flat}
    labels, v = s["labels"], case["v"]
    n, t = labels.shape
    live = (labels >= 0).flatten()
    rows = live.nonzero()[:, 0]
    flat = s["logits"].flatten(0, 1)
    logp = torch.zeros(n * t, dtype=f, device=DEV)
    for part in rows.split(max(1, (1 << 28) // v)):  # a part of the rows at a time: float64 rows are wide
        logp[part] = torch.log_softmax(flat[part].to(f), -1).gather(1, labels.flatten()[part][:, None])[:, 0]
    live = live.view(n, t)
    leaf = logp.view(n, t).clone().requires_grad_(True)
    counts = live.sum(-1).clamp(min=1).to(f)
    if case["op"] == "pref":
        gaps = ((leaf - s["ref_logp"].to(f)) * live).sum(-1)
        ratio = gaps / counts if case["average"] else gaps
        h = ratio[: n // 2] - ratio[n // 2:]
        if case["kind"] == "sigmoid":
            ls = torch.nn.functional.logsigmoid
            loss = -(1 - case["smoothing"]) * ls(BETA * h) - case["smoothing"] * ls(-BETA * h)
        elif case["kind"] == "hinge":
            loss = torch.relu(1 - BETA * h)
        else:
            loss = (h - 1 / (2 * BETA)) ** 2
        out, total = {"loss": loss.detach(), "logratio": ratio.detach()}, loss.mean()
    else:
        r = ((leaf - s["old_logp"].to(f)) * live).exp()
        a = s["advantages"].to(f)
        each = -torch.min(r * a, r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * a)
        kl = torch.zeros_like(each)
        if s["ref_logp"] is not None:
            q = (s["ref_logp"].to(f) - leaf) * live
            kl = q.exp() - q - 1
        share = live.to(f)
        share = share / share.sum() if case["reduction"] == "token" else share / counts[:, None] / n
        total = ((each + KL * kl) * share).sum()
        out = {"loss": total.detach(), "kl": (kl * share).sum().detach()}
    out["logp"] = logp.view(n, t)
    if case["step"] == "step":
        (slope,) = torch.autograd.grad(total, leaf)
        d = torch.zeros(n * t, v, dtype=f, device=DEV)
        for part in rows.split(max(1, (1 << 28) // v)):
            block = torch.softmax(flat[part].to(f), -1).neg_()
            block.scatter_add_(1, labels.flatten()[part][:, None], torch.ones(len(part), 1, dtype=f, device=DEV))
            d[part] = block.mul_(slope.flatten()[part][:, None])
        out["dlogits"] = d.view(n, t, v)
    return out
