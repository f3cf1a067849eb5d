"""fp64 oracle of the residual block's operators: layer norm, linear with bias,
activation and residual, gated feed-forward; forward and backward (numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Everything follows the
formulas in ``include/mamba3_ssm.h``; the matrix product and erf are the only
library steps.  Beside each result stands a bound of how far a computation
with fp32 sums may be from it (``u_out``: rounding of the outputs, ``u_dp``:
rounding of dP before the products), from the usual model: every operation's
relative error is at most one unit, 2^-23, and a sum of n terms is off by at
most n units of the sum of their magnitudes.
"""
import math

import numpy as np
from scipy.special import erf

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")
U32 = 2.0 ** -23
# largest |act'| of any activation (gelu: 1.129) and |act''| (relu excepted)
SLOPE, CURVE = 1.13, 1.0
# evaluation error of act and act' on top of that of its argument, of max(1, |z|):
# exponential, reciprocal, polynomial, product
ACT_EVAL = 2e-6


def act(z, name):
    if name == "relu":
        return np.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "sigmoid":
        return 1 / (1 + np.exp(-z))
    return z


def dact(z, name):
    if name == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if name in ("silu", "sigmoid"):
        p = 1 / (1 + np.exp(-z))
        return p * (1 - p) if name == "sigmoid" else p + z * p * (1 - p)
    if name == "gelu":
        return 0.5 * (1 + erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = np.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def layer_norm(x, gain, bias, eps):
    """(y, mean, rstd); gain, bias may be None."""
    mean = x.mean(1)
    z = x - mean[:, None]
    rstd = 1 / np.sqrt((z * z).mean(1) + eps)
    y = z * rstd[:, None]
    y = y if gain is None else y * gain
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_bound(x, gain, bias, eps, u_out):
    y, mean, rstd = layer_norm(x, gain, bias, eps)
    D = x.shape[1]
    c = (D + 32) * U32
    g = 1.0 if gain is None else np.abs(gain)
    b = 0.0 if bias is None else np.abs(bias)
    mag = np.abs(x).mean(1)
    # the mean is off by c mag; it moves every entry by that, and the spread by c of itself
    e_mean = c * mag
    e = g * (rstd[:, None] * e_mean[:, None] + c * np.abs((x - mean[:, None]) * rstd[:, None]) + 4 * U32) + 4 * U32 * b
    e_rstd = rstd * (2 * c + (rstd * e_mean) ** 2)
    return e * (1 + u_out) + u_out * np.abs(y) + 1e-30, e_mean + 1e-30, e_rstd


def layer_norm_bwd(x, gain, mean, rstd, dy, dskip=None):
    xh = (x - mean[:, None]) * rstd[:, None]
    a = dy if gain is None else dy * gain
    dx = rstd[:, None] * (a - a.mean(1, keepdims=True) - xh * (a * xh).mean(1, keepdims=True))
    return (dx if dskip is None else dx + dskip), (dy * xh).sum(0), dy.sum(0)


def layer_norm_bwd_bound(x, gain, mean, rstd, dy, dskip, u_out):
    M, D = x.shape
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    e_xh = 4 * U32 * (np.abs(x) + np.abs(mean)[:, None]) * rstd[:, None]
    a = np.abs(dy) if gain is None else np.abs(dy * gain)
    c = (D + 32) * U32
    m1, m2 = a.mean(1, keepdims=True), (a * xh).mean(1, keepdims=True)
    m2e = (a * e_xh).mean(1, keepdims=True)
    e = rstd[:, None] * (c * (a + m1 + xh * m2) + e_xh * m2 + xh * m2e)
    dx = np.abs(layer_norm_bwd(x, gain, mean, rstd, dy, dskip)[0])
    r = (M + 32) * U32
    return (e + 4 * U32 * dx + u_out * dx + 1e-30, r * (np.abs(dy) * xh).sum(0) + (np.abs(dy) * e_xh).sum(0) + 1e-30,
            r * np.abs(dy).sum(0) + 1e-30)


def _pre(x, W, bias):
    pre = x @ W.T
    e = (x.shape[1] + 16) * U32 * (np.abs(x) @ np.abs(W).T)
    if bias is not None:
        pre = pre + bias
        e = e + U32 * (np.abs(pre) + np.abs(bias))
    return pre, e


def linear(x, W, bias, residual, name):
    """(y, pre)"""
    pre, _ = _pre(x, W, bias)
    y = act(pre, name)
    return (y if residual is None else y + residual), pre


def linear_bound(x, W, bias, residual, name, u_out):
    pre, e = _pre(x, W, bias)
    y = np.abs(linear(x, W, bias, residual, name)[0])
    ey = SLOPE * e + (0 if name in ("none", "relu") else ACT_EVAL) * np.maximum(1, np.abs(pre)) + 2 * U32 * y
    return ey * (1 + u_out) + u_out * y + 1e-30, e * (1 + u_out) + u_out * np.abs(pre) + 1e-30


def gated(x, W, bias, name):
    """(h, pre)"""
    pre, _ = _pre(x, W, bias)
    F = W.shape[0] // 2
    return act(pre[:, :F], name) * pre[:, F:], pre


def gated_bound(x, W, bias, name, u_out):
    pre, e = _pre(x, W, bias)
    F = W.shape[0] // 2
    g, u = pre[:, :F], pre[:, F:]
    ef = SLOPE * e[:, :F] + (0 if name in ("none", "relu") else ACT_EVAL) * np.maximum(1, np.abs(g))
    h = np.abs(act(g, name) * u)
    eh = ef * (np.abs(u) + e[:, F:]) + np.abs(act(g, name)) * e[:, F:] + 2 * U32 * h
    return eh * (1 + u_out) + u_out * h + 1e-30, e * (1 + u_out) + u_out * np.abs(pre) + 1e-30


def dp_linear(pre, dy, name):
    return dy if name == "none" else dy * dact(pre, name)


def dp_gated(pre, dy, name):
    F = pre.shape[1] // 2
    g, u = pre[:, :F], pre[:, F:]
    return np.concatenate([dy * u * dact(g, name), dy * act(g, name)], 1)


def dp_eval(pre, dy, name, is_gated):
    """Error of dP before any rounding to the io type."""
    k = 0 if name in ("none", "relu") else ACT_EVAL
    if not is_gated:
        return np.abs(dy) * (k * np.maximum(1, np.abs(pre)) + 2 * U32) if pre is not None else 0 * np.abs(dy)
    F = pre.shape[1] // 2
    g, u = np.abs(pre[:, :F]), np.abs(pre[:, F:])
    d = np.abs(dy)
    z = np.maximum(1, g) * (k + 4 * U32)
    return np.concatenate([d * u * z, d * z], 1)


def products(dp, x, W):
    """dx, dW, dbias from dP."""
    return dp @ W, dp.T @ x, dp.sum(0)


def products_bound(dp, e_dp, x, W, u_out, u_dp):
    """e_dp: error of dP before its rounding (u_dp)."""
    M, N = dp.shape
    a = np.abs(dp)
    ed = e_dp + u_dp * (a + e_dp)  # what the products take
    aW, ax = np.abs(W), np.abs(x)
    dx, dW, db = products(dp, x, W)
    ex = ed @ aW + (N + 16) * U32 * (a + ed) @ aW
    ew = ed.T @ ax + (M + 16) * U32 * (a + ed).T @ ax
    eb = e_dp.sum(0) + (M + 16) * U32 * a.sum(0)
    return (ex * (1 + u_out) + u_out * np.abs(dx) + 1e-30, ew * (1 + u_out) + u_out * np.abs(dW) + 1e-30, eb + 1e-30)
