"""fp64 oracle of the attention layer's operators: norms of queries and keys
with rotation, windowed attention with sinks, forward and backward, and that
over a cache (numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Everything follows the
formulas in ``include/mamba3_ssm.h``.  Beside each result stands a bound of how
far a computation with fp32 sums may be from it (``u_out``: rounding of the
outputs, ``u_mid``: rounding of p and ds as operands of the products that take
them; half a step of their type each, relative), from the usual model: every
fp32 operation is off by at most one unit, 2^-23, relatively, and a sum of n
terms by at most n units of the sum of their magnitudes.
"""
import numpy as np

U32 = 2.0 ** -23


# --------------------------------------------------------------------------
# norms of heads with rotation
# --------------------------------------------------------------------------
def _pairs(D, R, halves):
    """Indices of the pairs' first and second entries."""
    j = np.arange(R // 2)
    return (j, j + R // 2) if halves else (2 * j, 2 * j + 1)


def rotate(z, theta, pos, halves, sign=1.0):
    """z (rows, heads, D) with pair j of row r turned by sign pos[r] theta[j]."""
    R = 0 if theta is None else 2 * len(theta)
    out = z.copy()
    if R == 0:
        return out
    a, b = _pairs(z.shape[-1], R, halves)
    w = pos.astype(np.float64)[:, None, None] * theta
    c, s = np.cos(w), sign * np.sin(w)
    out[..., a] = z[..., a] * c - z[..., b] * s
    out[..., b] = z[..., a] * s + z[..., b] * c
    return out


def _reach(z, theta, halves):
    """|a| + |b| of the pair an entry belongs to (its own magnitude without one)."""
    R = 0 if theta is None else 2 * len(theta)
    m = np.abs(z)
    out = m.copy()
    if R:
        a, b = _pairs(z.shape[-1], R, halves)
        out[..., a] = out[..., b] = m[..., a] + m[..., b]
    return out


def norm_rope(x, gain, eps, theta, pos, halves):
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = x * r if gain is None else x * r * gain
    return rotate(z, theta, pos, halves)


def norm_rope_bound(x, gain, eps, theta, pos, halves, u_out):
    # r is off by (D + 16) / 2 units, cosines and sines by 4 units absolutely
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = x * r if gain is None else x * r * gain
    e = ((x.shape[-1] + 16) / 2 + 12) * U32 * _reach(z, theta, halves)
    return e * (1 + u_out) + u_out * np.abs(rotate(z, theta, pos, halves)) + 1e-30


def norm_rope_bwd(x, gain, eps, theta, pos, halves, dy):
    """(dx, dgain)"""
    dz = rotate(dy, theta, pos, halves, -1.0)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    a = dz if gain is None else dz * gain
    return r * (a - xh * (a * xh).mean(-1, keepdims=True)), (dz * xh).sum((0, 1))


def norm_rope_bwd_bound(x, gain, eps, theta, pos, halves, dy, u_out):
    D = x.shape[-1]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = np.abs(x * r)
    g = 1.0 if gain is None else np.abs(gain)
    dz = _reach(dy, theta, halves)
    c = ((D + 16) / 2 + 12) * U32
    m = (dz * g * xh).mean(-1, keepdims=True)
    e = r * (c * dz * g + xh * m * (D + 16 + 4 * (D + 16) / 2) * U32 + 4 * U32 * (dz * g + xh * m))
    dx = np.abs(norm_rope_bwd(x, gain, eps, theta, pos, halves, dy)[0])
    n = x.shape[0] * x.shape[1]
    return (e * (1 + u_out) + u_out * dx + 1e-30, ((n + 16) * U32 + c) * (dz * xh).sum((0, 1)) + 1e-30)


# --------------------------------------------------------------------------
# attention of one sequence: q (n, Hq, D), k and v (m, Hk, D)
# --------------------------------------------------------------------------
def visible(n, m, window, sinks):
    p, j = (m - n + np.arange(n))[:, None], np.arange(m)[None]
    see = j <= p
    return see & ((p - j < window) | (j < sinks)) if window else see


def _heads(x, Hq):
    """(m, Hk, D) -> (Hq, m, D), each head for those that share it."""
    return np.repeat(x.transpose(1, 0, 2), Hq // x.shape[1], axis=0)


def _scores(q, k, scale, see):
    """Scores (Hq, n, m), -inf where nothing is seen, and their bound."""
    Q, K = q.transpose(1, 0, 2), _heads(k, q.shape[1])
    s = scale * Q @ K.transpose(0, 2, 1)
    e = (q.shape[2] + 16) * U32 * scale * (np.abs(Q) @ np.abs(K).transpose(0, 2, 1))
    return np.where(see, s, -np.inf), np.where(see, e, 0.0)


def attention(q, k, v, window, sinks, scale, see=None):
    """(o (n, Hq, D), lse (n, Hq))"""
    see = visible(len(q), len(k), window, sinks) if see is None else see
    s, _ = _scores(q, k, scale, see)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.exp(s - np.where(m == -np.inf, 0.0, m))
    total = p.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(total))[..., 0]
    o = p @ _heads(v, q.shape[1]) / np.where(total == 0, 1.0, total)
    return o.transpose(1, 0, 2), lse.T


def attention_bound(q, k, v, window, sinks, scale, u_out, u_mid, see=None):
    """Bounds of o and lse."""
    n, m = len(q), len(k)
    see = visible(n, m, window, sinks) if see is None else see
    s, e = _scores(q, k, scale, see)
    o, lse = attention(q, k, v, window, sinks, scale, see)
    top = np.where(see, np.abs(s), 0.0).max(-1, keepdims=True, initial=0.0)
    w = np.exp(s - np.where(lse.T == -np.inf, 0.0, lse.T)[..., None])
    # an exponent is a product, a difference and an exponential away from its
    # score; the reference m it is taken from may lie 12 powers of two behind the
    # maximum, 8.4 in natural units: |m| <= top + 8.4 and |s - m| <= |s| + top + 8.4.
    # Both are off by a unit at most, the scale's factor by another of |s - m|, the
    # exponential by one: U32 (2 |s| + 3 top + 26.2) in all, within the four units here
    e = e + np.where(see, 4 * U32 * (np.abs(np.where(see, s, 0.0)) + top + 8), 0.0)
    mean = (w * e).sum(-1, keepdims=True)
    V = np.abs(_heads(v, q.shape[1]))
    # weights off by e and their sum by its mean, one rounding of each weight,
    # sums over the keys with a rescaling now and then
    eo = (w * (e + mean + u_mid + (m + 64) * U32)) @ V
    eo = eo.transpose(1, 0, 2)
    el = (mean + (m + 64) * U32)[..., 0].T + 4 * U32 * np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return eo * (1 + u_out) + u_out * np.abs(o) + 1e-30, el + 1e-30


def attention_bwd(q, k, v, o, lse, do, window, sinks, scale):
    """(dq, dk, dv) from o and lse as given."""
    return _attention_bwd(q, k, v, o, lse, do, window, sinks, scale, None, None)[0]


def attention_bwd_bound(q, k, v, o, lse, do, window, sinks, scale, u_out, u_mid):
    return _attention_bwd(q, k, v, o, lse, do, window, sinks, scale, u_out, u_mid)[1]


def _attention_bwd(q, k, v, o, lse, do, window, sinks, scale, u_out, u_mid):
    n, Hq, D = q.shape
    m, Hk = k.shape[:2]
    see = visible(n, m, window, sinks)
    s, e = _scores(q, k, scale, see)
    l = lse.T[..., None]
    p = np.where(see & (l > -np.inf), np.exp(s - np.where(l > -np.inf, l, 0.0)), 0.0)
    dO, V, Q, K = do.transpose(1, 0, 2), _heads(v, Hq), q.transpose(1, 0, 2), _heads(k, Hq)
    dp = dO @ V.transpose(0, 2, 1)
    delta = (do * o).sum(-1).T[..., None]
    ds = p * (dp - delta)

    def shared(x):  # (Hq, m, D): summed over the heads that share one
        return x.reshape(Hk, Hq // Hk, m, D).sum(1).transpose(1, 0, 2)

    grads = (scale * (ds @ K).transpose(1, 0, 2), scale * shared(ds.transpose(0, 2, 1) @ Q),
             shared(p.transpose(0, 2, 1) @ dO))
    if u_out is None:
        return grads, None
    aQ, aK, aV, aO = (np.abs(x) for x in (Q, K, V, dO))
    c = (D + 16) * U32
    ep = p * (e + np.where(see, 4 * U32 * (np.abs(np.where(see, s, 0.0)) + np.abs(np.where(np.isfinite(l), l, 0.0)) + 1), 0.0))
    e_dp = c * (aO @ aV.transpose(0, 2, 1)) + c * (np.abs(do) * np.abs(o)).sum(-1).T[..., None]
    eds = p * e_dp + ep * (np.abs(dp - delta) + e_dp) + 3 * U32 * np.abs(ds)
    ap, ads = np.abs(p), np.abs(ds)
    tp, tds = ep + u_mid * (ap + ep), eds + u_mid * (ads + eds)
    G = Hq // Hk
    eq = scale * ((tds + (m + 64) * U32 * (ads + tds)) @ aK).transpose(1, 0, 2)
    ek = scale * shared((tds + (n * G + 64) * U32 * (ads + tds)).transpose(0, 2, 1) @ aQ)
    ev = shared((tp + (n * G + 64) * U32 * (ap + tp)).transpose(0, 2, 1) @ aO)
    return grads, tuple(x * (1 + u_out) + u_out * np.abs(g) + 4 * U32 * np.abs(g) + 1e-30
                        for x, g in zip((eq, ek, ev), grads))


# --------------------------------------------------------------------------
# attention over a cache: the whole sequences are told, and what the cache
# still holds of them is seen
# --------------------------------------------------------------------------
def slot(p, sinks, capacity):
    return p if p < sinks else sinks + (p - sinks) % (capacity - sinks)


def held(total, sinks, capacity):
    """Positions of the tokens that a cache holds after `total` of them."""
    ring = capacity - sinks
    return [p for p in range(total) if p < sinks or p >= max(sinks, total - ring)]


def decode_visible(total, tokens, window, sinks, capacity):
    """(T, total): which of all tokens the last T see."""
    see = visible(tokens, total, window, sinks)
    there = np.zeros(total, dtype=bool)
    there[held(total, sinks, capacity)] = True
    return see & there[None]
