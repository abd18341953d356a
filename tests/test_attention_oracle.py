"""Pins of the sublayer oracle: known answers, other routes to the same values, differences."""

from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import attention_oracle as ao


def test_philox_known_answers():
    # the published test vectors of Philox4x32-10
    ones = 0xFFFFFFFF
    cases = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
             ((ones,) * 4, (ones,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
              (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for counter, key, want in cases:
        assert tuple(int(x) for x in ao.philox([counter], key)[0]) == want


def test_dropout_rate_and_mean():
    keep, scale = ao.dropout_keep(1 << 20, 0.3, 7, 9)
    least = round(0.3 * 65536)
    # a binomial share: five standard deviations
    assert abs(keep.mean() - (1 - least / 65536)) < 5 * math.sqrt(0.3 * 0.7 / (1 << 20))
    assert scale * (1 - least / 65536) == 1.0
    assert not np.array_equal(keep, ao.dropout_keep(1 << 20, 0.3, 7, 10)[0])
    assert ao.dropout_keep(100, 1.0, 1, 0)[1] == 0.0 and not ao.dropout_keep(100, 1.0, 1, 0)[0].any()
    assert ao.dropout_keep(100, 0.0, 1, 0)[0].all()


def test_buckets():
    # by hand: 32 two-sided buckets to 128: 8 exact ones a side, then doubling every two buckets
    got = [ao.bucket(-n, 32, 128, True) for n in (0, 1, 7, 8, 11, 12, 15, 16, 23, 32, 64, 91, 127, 128, 10**6)]
    assert got == [0, 1, 7, 8, 8, 9, 9, 10, 11, 12, 14, 15, 15, 15, 15]
    assert [ao.bucket(n, 32, 128, True) for n in (1, 7, 8, 128)] == [17, 23, 24, 31]
    assert [ao.bucket(n, 32, 128, False) for n in (5, 0, -1, -15, -16, -128)] == [0, 0, 1, 15, 16, 31]
    for count, distance in ((32, 128), (7, 64), (45, 500)):
        for n in range(1, 600):
            small = count // 2
            x = math.log(n / small) / math.log(distance / small) * (count - small) if n >= small else 0.0
            if n >= small and abs(x - round(x)) > 1e-9:
                assert ao.bucket(-n, count, distance, False) == min(count - 1, small + math.floor(x)), (count, n)


def test_bias_gradient_is_the_adjoint():
    r = np.random.default_rng(0)
    table, up = r.standard_normal((8, 3)), r.standard_normal((2, 3, 9, 11))
    bias = ao.relative_bias(table, 9, 11, 20, True)
    np.testing.assert_allclose((bias[None] * up).sum(), (table * ao.relative_bias_bwd(up, 8, 20, True)).sum(),
                               rtol=1e-12)


@pytest.mark.parametrize("causal,spans,biased", [(0, 0, 0), (1, 0, 1), (0, 1, 1), (1, 1, 0)])
def test_attention_gradients_against_differences(causal, spans, biased):
    r = np.random.default_rng(1)
    b, tq, tk, h, hk, d = 2, 5, 7, 4, 2, 3
    q, k, v = r.standard_normal((b, tq, h, d)), r.standard_normal((b, tk, hk, d)), r.standard_normal((b, tk, hk, d))
    up = r.standard_normal(q.shape)
    table = r.standard_normal((8, h))
    see = ao.visible(b, tq, tk, bool(causal), [1, 0] if spans else None, [4, 0] if spans else None)

    def loss(q, k, v, table):
        bias = ao.relative_bias(table, tq, tk, 20, True) if biased else None
        return (ao.attention(q, k, v, 0.7, see, bias)[0] * up).sum()

    bias = ao.relative_bias(table, tq, tk, 20, True) if biased else None
    _, _, p = ao.attention(q, k, v, 0.7, see, bias)
    dq, dk, dv, ds = ao.attention_bwd(q, k, v, p, up, 0.7)
    args, eps = [q, k, v, table], 1e-5
    grads = [dq, dk, dv, ao.relative_bias_bwd(ds, 8, 20, True)] if biased else [dq, dk, dv]
    for n, g in enumerate(grads):
        for _ in range(6):
            at = tuple(r.integers(0, s) for s in args[n].shape)
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[n][at] += eps
            lo[n][at] -= eps
            # central differences: eps^2 times the third derivative, and rounding / eps
            assert abs((loss(*hi) - loss(*lo)) / (2 * eps) - g[at]) < 1e-8


def test_attention_by_hand():
    # one query, two keys with scores log 3 and 0
    q, k = np.array([[[[1.0]]]]), np.array([[[[math.log(3)]], [[0.0]]]])
    v = np.array([[[[4.0]], [[8.0]]]])
    o, lse, p = ao.attention(q, k, v, 1.0, ao.visible(1, 1, 2))
    np.testing.assert_allclose([o[0, 0, 0, 0], lse[0, 0, 0]], [5.0, math.log(4)], rtol=1e-14)
    o, lse, p = ao.attention(q, k, v, 1.0, ao.visible(1, 1, 2, end=[0]))
    assert o.item() == 0 and lse.item() == -np.inf and not p.any()
