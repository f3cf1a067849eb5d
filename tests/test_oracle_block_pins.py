"""Pins of the residual block's fp64 oracle (oracle/block.py): hand-computed
values, the activations' identities, and every gradient against central
differences of the forward; planted mistakes have to be caught by them."""
import math

import numpy as np
import pytest

from oracle import block

RNG = np.random.default_rng


def differences(f, a, d, h=1e-5):
    """sum(d * f) differentiated by every entry of a."""
    g = np.zeros_like(a)
    it = np.nditer(a, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = a[i]
        a[i] = old + h
        up = (d * f()).sum()
        a[i] = old - h
        g[i] = (up - (d * f()).sum()) / (2 * h)
        a[i] = old
    return g


def close(a, b, tol=1e-8):
    return np.max(np.abs(a - b)) <= tol * max(1.0, np.max(np.abs(b)))


def test_layer_norm_by_hand():
    # (1, 3): mean 2, variance 1; eps = 3 gives rstd 1/2
    y, mean, rstd = block.layer_norm(np.array([[1.0, 3.0]]), np.array([2.0, 4.0]), np.array([0.5, -1.0]), 3.0)
    assert mean[0] == 2.0 and rstd[0] == 0.5
    assert np.array_equal(y, [[-0.5, 1.0]])
    # a constant row: only the bias is left
    y, _, _ = block.layer_norm(np.full((1, 5), 7.0), None, np.arange(5.0), 1e-5)
    assert np.array_equal(y[0], np.arange(5.0))


@pytest.mark.parametrize("name,at1", [("none", 1.0), ("relu", 1.0), ("silu", 1 / (1 + math.exp(-1))),
                                      ("gelu", 0.8413447460685429), ("gelu_tanh", 0.8411919906082768),
                                      ("sigmoid", 1 / (1 + math.exp(-1)))])
def test_activations(name, at1):
    z = np.linspace(-4, 4, 41)
    assert abs(block.act(np.array([1.0]), name)[0] - at1) < 1e-12
    zz = z[np.abs(z) > 1e-3]  # relu has no derivative at 0
    d = (block.act(zz + 1e-6, name) - block.act(zz - 1e-6, name)) / 2e-6
    assert close(block.dact(zz, name), d, 1e-8)
    assert np.all(np.abs(block.dact(z, name)) <= block.SLOPE)
    if name in ("silu", "gelu", "gelu_tanh"):  # z and its mirror differ by z
        assert np.allclose(block.act(z, name) - block.act(-z, name), z, atol=1e-12)


@pytest.mark.parametrize("seed", [0, 1])
def test_layer_norm_gradient_matches_differences(seed):
    r = RNG(seed)
    x, gain, bias = r.standard_normal((3, 7)), r.standard_normal(7), r.standard_normal(7)
    dy, skip = r.standard_normal((3, 7)), r.standard_normal((3, 7))
    f = lambda: block.layer_norm(x, gain, bias, 1e-3)[0]
    _, mean, rstd = block.layer_norm(x, gain, bias, 1e-3)
    dx, dg, db = block.layer_norm_bwd(x, gain, mean, rstd, dy, skip)
    assert close(dx - skip, differences(f, x, dy))
    assert close(dg, differences(f, gain, dy)) and close(db, differences(f, bias, dy))
    # planted mistakes: without the mean of a, or without the mean of a xh
    xh, a = (x - mean[:, None]) * rstd[:, None], dy * gain
    assert not close(rstd[:, None] * (a - xh * (a * xh).mean(1, keepdims=True)), differences(f, x, dy), 1e-4)
    assert not close(rstd[:, None] * (a - a.mean(1, keepdims=True)), differences(f, x, dy), 1e-4)


@pytest.mark.parametrize("name", block.ACTS)
@pytest.mark.parametrize("is_gated", [False, True])
def test_product_gradients_match_differences(name, is_gated):
    r = RNG(3)
    x, W, bias = r.standard_normal((4, 5)), r.standard_normal((6, 5)), r.standard_normal(6)
    n = 3 if is_gated else 6
    dy = r.standard_normal((4, n))
    if is_gated:
        f = lambda: block.gated(x, W, bias, name)[0]
        dp = block.dp_gated(block.gated(x, W, bias, name)[1], dy, name)
    else:
        res = r.standard_normal((4, 6))
        f = lambda: block.linear(x, W, bias, res, name)[0]
        dp = block.dp_linear(block.linear(x, W, bias, res, name)[1], dy, name)
        assert close(differences(f, res, dy), dy)
    dx, dW, db = block.products(dp, x, W)
    assert close(dx, differences(f, x, dy)) and close(dW, differences(f, W, dy)) and close(db, differences(f, bias, dy))
    if is_gated:  # planted: the gate's and the other half's gradients exchanged
        assert not close(block.products(np.roll(dp, 3, 1), x, W)[0], dx, 1e-3)


def test_gated_by_hand():
    # one entry, W picks g = x0, u = x1: h = relu(2) * 3
    h, pre = block.gated(np.array([[2.0, 3.0]]), np.eye(2), None, "relu")
    assert h[0, 0] == 6.0 and np.array_equal(pre, [[2.0, 3.0]])
