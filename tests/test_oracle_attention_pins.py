"""Pins of oracle/attention.py: hand-computed values, an independent
formulation of each operator, and central differences of the forwards."""
import math

import numpy as np
import pytest

from oracle import attention as oracle


def test_norm_rope_by_hand():
    # a head of (3, 4) has mean square 12.5; a quarter turn maps (a, b) to (-b, a)
    x = np.array([[[3.0, 4.0]]])
    got = oracle.norm_rope(x, None, 0.0, np.array([1.0]), np.array([math.pi / 2]), False)
    assert np.allclose(got, np.array([-4.0, 3.0]) / math.sqrt(12.5), atol=1e-15)
    got = oracle.norm_rope(x, np.array([2.0, 1.0]), 12.5, None, np.array([7]), False)
    assert np.allclose(got, np.array([6.0, 4.0]) / 5.0, atol=1e-15)
    # pairs: (0, 2), (1, 3) half apart, the rest not turned
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    got = oracle.rotate(x, np.array([0.0, math.pi]), np.array([1]), True)
    assert np.allclose(got, [[[1.0, -2.0, 3.0, -4.0, 5.0]]], atol=1e-15)


@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope_as_complex_numbers(halves):
    r = np.random.default_rng(0)
    x, gain, theta, pos = r.standard_normal((6, 3, 10)), r.standard_normal(10), r.standard_normal(4), r.integers(-50, 50, 6)
    z = x / np.sqrt((x ** 2).sum(-1, keepdims=True) / 10 + 0.1) * gain
    c = z[..., :4] + 1j * z[..., 4:8] if halves else z[..., 0:8:2] + 1j * z[..., 1:8:2]
    c = c * np.exp(1j * pos[:, None, None] * theta)
    want = z.copy()
    if halves:
        want[..., :4], want[..., 4:8] = c.real, c.imag
    else:
        want[..., 0:8:2], want[..., 1:8:2] = c.real, c.imag
    assert np.allclose(oracle.norm_rope(x, gain, 0.1, theta, pos, halves), want, atol=1e-14)


def quotient(f, args, i, at, step=1e-5):
    up, down = [[a.copy() for a in args] for _ in range(2)]
    up[i][at] += step
    down[i][at] -= step
    return (f(*up) - f(*down)) / (2 * step)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("pairs", [0, 3, 4])
def test_norm_rope_gradients(halves, pairs):
    r = np.random.default_rng(1)
    x, gain, dy = r.standard_normal((3, 2, 8)), r.standard_normal(8), r.standard_normal((3, 2, 8))
    theta = r.standard_normal(pairs) if pairs else None
    pos = np.array([5, 0, -3])
    f = lambda x, g: float((oracle.norm_rope(x, g, 0.1, theta, pos, halves) * dy).sum())
    dx, dgain = oracle.norm_rope_bwd(x, gain, 0.1, theta, pos, halves, dy)
    for i, d in enumerate((dx, dgain)):
        for at in np.ndindex(*d.shape):
            assert abs(quotient(f, (x, gain), i, at) - d[at]) < 1e-8


def attend(q, k, v, window, sinks, scale):
    """One query, key and head at a time."""
    n, Hq, D = q.shape
    m, Hk = k.shape[:2]
    o, lse = np.zeros_like(q), np.full((n, Hq), -np.inf)
    for i in range(n):
        p = m - n + i
        for h in range(Hq):
            kh = h // (Hq // Hk)
            js = [j for j in range(m) if j <= p and (window == 0 or p - j < window or j < sinks)]
            if js:
                w = [math.exp(scale * sum(q[i, h, d] * k[j, kh, d] for d in range(D))) for j in js]
                lse[i, h] = math.log(sum(w))
                o[i, h] = sum(x * v[j, kh] for x, j in zip(w, js)) / sum(w)
    return o, lse


@pytest.mark.parametrize("n,m,window,sinks", [(6, 6, 0, 0), (6, 6, 2, 0), (6, 6, 2, 1), (3, 8, 3, 2), (8, 3, 2, 1), (5, 5, 1, 9)])
def test_attention_pair_by_pair(n, m, window, sinks):
    r = np.random.default_rng(n + m)
    q, k, v = r.standard_normal((n, 4, 3)), r.standard_normal((m, 2, 3)), r.standard_normal((m, 2, 3))
    for got, want in zip(oracle.attention(q, k, v, window, sinks, 0.7), attend(q, k, v, window, sinks, 0.7)):
        assert np.allclose(got, want, atol=1e-13)


@pytest.mark.parametrize("n,m,window,sinks", [(5, 5, 0, 0), (5, 5, 2, 1), (3, 6, 2, 1), (6, 3, 2, 1)])
def test_attention_gradients(n, m, window, sinks):
    r = np.random.default_rng(n * m)
    q, k, v = r.standard_normal((n, 4, 3)), r.standard_normal((m, 2, 3)), r.standard_normal((m, 2, 3))
    do = r.standard_normal((n, 4, 3))
    o, lse = oracle.attention(q, k, v, window, sinks, 0.7)
    f = lambda q, k, v: float((oracle.attention(q, k, v, window, sinks, 0.7)[0] * do).sum())
    for i, d in enumerate(oracle.attention_bwd(q, k, v, o, lse, do, window, sinks, 0.7)):
        for at in np.ndindex(*d.shape):
            assert abs(quotient(f, (q, k, v), i, at) - d[at]) < 1e-8, (i, at)


def test_cache_told_from_its_beginning():
    # slots written token by token hold what held() says, each at its slot
    for sinks, capacity in ((0, 5), (2, 7), (3, 4)):
        slots = [None] * capacity
        for p in range(23):
            slots[oracle.slot(p, sinks, capacity)] = p
            assert sorted(x for x in slots if x is not None) == oracle.held(p + 1, sinks, capacity)


def test_bounds_are_of_the_roundings_size():
    # not so wide that a wrong result would pass: bf16's bounds stay within a few
    # half steps of the outputs' typical size, fp32's within a thousandth of those
    r = np.random.default_rng(2)
    q, k, v = r.standard_normal((60, 2, 64)), r.standard_normal((60, 1, 64)), r.standard_normal((60, 1, 64))
    o, lse = oracle.attention(q, k, v, 20, 2, 0.125)
    do = r.standard_normal(o.shape)
    for u, most in ((2.0 ** -8, 0.02), (2.0 ** -24, 2e-4)):
        b, _ = oracle.attention_bound(q, k, v, 20, 2, 0.125, u, u)
        assert np.median(b) < most * np.abs(v).mean()
        g = oracle.attention_bwd(q, k, v, o, lse, do, 20, 2, 0.125)
        for x, e in zip(g, oracle.attention_bwd_bound(q, k, v, o, lse, do, 20, 2, 0.125, u, u)):
            assert np.median(e) < 4 * most * np.abs(x).max()
        x = r.standard_normal((30, 2, 64))
        a = (x, None, 1e-5, np.ones(32), np.arange(30), False)
        assert np.median(oracle.norm_rope_bound(*a, u)) < most
        for w, e in zip(oracle.norm_rope_bwd(*a, x[::-1]), oracle.norm_rope_bwd_bound(*a, x[::-1], u)):
            assert np.median(e) < 4 * most * np.abs(w).max()
