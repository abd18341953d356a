"""float64 oracle of a sublayer's operators (numpy, test infrastructure only).

Attention and its gradients, the relative position bias by buckets and dropout
from Philox4x32-10, each the formula written out; nothing here is shared with
the HIP path.
"""

from __future__ import annotations

import numpy as np


def bucket(rel: int, count: int, max_distance: int, two_sided: bool) -> int:
    """The bucket of a relative position, in whole numbers: the logarithm's
    floor is at least m where (n / small)^rest >= (max_distance / small)^m."""
    side, base = (count // 2, count // 2 if rel > 0 else 0) if two_sided else (count, 0)
    n = abs(rel) if two_sided else max(-rel, 0)
    small = side // 2
    if n < small:
        return base + n
    rest, m = side - small, 0
    while m + 1 < rest and n**rest * small ** (m + 1) >= max_distance ** (m + 1) * small**rest:
        m += 1
    return base + small + m


def bucket_matrix(tq, tk, count, max_distance, two_sided):
    one = {r: bucket(r, count, max_distance, two_sided) for r in range(-tq - tk, tq + tk + 1)}
    return np.array([[one[j - (i + tk - tq)] for j in range(tk)] for i in range(tq)], dtype=int).reshape(tq, tk)


def relative_bias(table, tq, tk, max_distance, two_sided):
    return table[bucket_matrix(tq, tk, table.shape[0], max_distance, two_sided)].transpose(2, 0, 1)


def relative_bias_bwd(dbias, count, max_distance, two_sided):
    """dtable (count, heads) of dbias (batch, heads, queries, keys)."""
    where = bucket_matrix(*dbias.shape[2:], count, max_distance, two_sided)
    out = np.zeros((count, dbias.shape[1]))
    for c in range(count):
        out[c] = dbias[:, :, where == c].sum(axis=(0, 2))
    return out


def visible(b, tq, tk, causal=False, begin=None, end=None):
    """(b, tq, tk): whether a query sees a key."""
    i, j = np.arange(tq)[:, None], np.arange(tk)[None, :]
    see = np.broadcast_to(j <= i + tk - tq if causal else np.ones((tq, tk), bool), (b, tq, tk)).copy()
    if begin is not None:
        see &= j[None] >= np.asarray(begin)[:, None, None]
    if end is not None:
        see &= j[None] < np.asarray(end)[:, None, None]
    return see


def attention(q, k, v, scale, see, bias=None):
    """(o, lse, p) of q (b, tq, h, d), k and v (b, tk, hk, d); bias (h, tq, tk)."""
    g = q.shape[2] // k.shape[2]
    kk, vv = np.repeat(k, g, axis=2), np.repeat(v, g, axis=2)
    s = np.matmul(q.transpose(0, 2, 1, 3), kk.transpose(0, 2, 3, 1)) * scale
    if bias is not None:
        s = s + bias
    s = np.where(see[:, None], s, -np.inf)
    with np.errstate(all="ignore"):
        top = s.max(-1, keepdims=True, initial=-np.inf)
        top = np.where(np.isfinite(top), top, 0.0)
        e = np.exp(s - top)
        total = e.sum(-1, keepdims=True)
        p = np.where(total > 0, e / np.where(total > 0, total, 1.0), 0.0)
        lse = np.where(total > 0, top + np.log(total), -np.inf)[..., 0]
    o = np.matmul(p, vv.transpose(0, 2, 1, 3)).transpose(0, 2, 1, 3)
    return o, lse, p


def attention_bwd(q, k, v, p, dout, scale):
    """(dq, dk, dv, ds) from the probabilities (b, h, tq, tk)."""
    b, tq, h, d = q.shape
    hk, g = k.shape[2], q.shape[2] // k.shape[2]
    kk, vv = (np.repeat(t, g, axis=2).transpose(0, 2, 1, 3) for t in (k, v))
    qq, do = q.transpose(0, 2, 1, 3), dout.transpose(0, 2, 1, 3)
    dp = np.matmul(do, vv.transpose(0, 1, 3, 2))
    ds = p * (dp - (p * dp).sum(-1, keepdims=True))
    dq = scale * np.matmul(ds, kk)

    def shared(t):  # summed over the heads that share a key head
        return t.reshape(b, hk, g, -1, d).sum(2).transpose(0, 2, 1, 3)

    dk = shared(scale * np.matmul(ds.transpose(0, 1, 3, 2), qq))
    dv = shared(np.matmul(p.transpose(0, 1, 3, 2), do))
    return dq.transpose(0, 2, 1, 3), dk, dv, ds


def philox(counter, key):
    """Philox4x32-10: counter (n, 4) and key (2) of 32-bit words -> (n, 4)."""
    c = [np.asarray(counter, np.uint64)[:, w].copy() for w in range(4)]
    k = [int(key[0]), int(key[1])]
    low, up = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> up) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> up) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).astype(np.uint32)


def dropout_keep(n, p, seed, offset):
    """Which of n elements are kept, and their scale."""
    blocks = np.arange(-(-n // 8), dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    ones = np.ones_like(blocks)
    counter = np.stack([blocks & low, blocks >> np.uint64(32), ones * np.uint64(offset & 0xFFFFFFFF),
                        ones * np.uint64(offset >> 32)], 1)
    words = philox(counter, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([words & 0xFFFF, words >> 16], -1).reshape(-1)[:n]
    least = int(np.rint(p * 65536))
    return bits >= least, 65536 / (65536 - least) if least < 65536 else 0.0


def dropout(x, p, seed, offset, residual=None):
    keep, scale = dropout_keep(x.size, p, seed, offset)
    y = np.where(keep.reshape(x.shape), x * scale, 0.0)
    return y if residual is None else y + residual
