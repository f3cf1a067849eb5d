"""Activations of the residual block's products and their derivatives, far from
zero relative to their own size, and at their ends.  Needs an MI355X.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -23


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from state_space_sequence_03_amd import ops as o
    o.lib()
    return o


TAILS = [(io, name, far) for name, far in (("sigmoid", 40.0), ("silu", 40.0), ("gelu", 12.0), ("gelu_tanh", 9.0))
         for io in ("bf16", "f32")]


def exact(z, name):
    """act(z) and act'(z) in 64 bits, without cancellation in the tails."""
    e = np.exp(-np.abs(z))
    p = np.where(z < 0, e, 1.0) / (1 + e)  # sigmoid
    if name == "sigmoid":
        return p, e / (1 + e) ** 2
    if name == "silu":
        return z * p, p * (1 + z * np.where(z < 0, 1.0, e) / (1 + e))
    if name == "gelu":
        phi = 0.5 * np.array([math.erfc(-v / math.sqrt(2)) for v in z])
        return z * phi, phi + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    s = 2 * a * (z + 0.044715 * z ** 3)
    e = np.exp(-np.abs(s))
    p, q = np.where(z < 0, e, 1.0) / (1 + e), np.where(z < 0, 1.0, e) / (1 + e)
    return z * p, p * (1 + z * q * 2 * a * (1 + 3 * 0.044715 * z * z))


def bound(z, name, io):
    """Relative error of act and act' at |z| >= 5.

    An exponential is off by the rounding of its argument m (U |m| for each
    rounding of it, of which there are at most 7, 2, 1) and a few units; a
    reciprocal and each product by a unit or two.  In act' two terms of opposite
    sign meet for z < 0: at |z| >= 5 that costs at most 1.5 for silu (1 + |z|
    over |z| - 1) and 1.1 for the others.  bf16 gelu takes Phi from a fit whose
    own relative error is 7e-7.  The results leave in fp32."""
    m = np.abs(z)
    if name in ("sigmoid", "silu"):
        return 2 * (m + 12) * U
    if name == "gelu":
        return 1.2 * ((m * m + 24) * U + (7e-7 if io == "bf16" else 0.0))
    return 1.2 * (7 * 2 * 0.7978845608 * m * (1 + 0.044715 * m * m) + 24) * U


@pytest.mark.parametrize("io,name,far", TAILS)
def test_tails_of_the_activations(ops, io, name, far):
    # one row: the bias' gradient is dP itself, in fp32, not rounded to the io type
    z = torch.linspace(5, far, 257).to(IO[io])
    z = torch.cat([z, -z]).cuda()
    n = z.numel()
    code = getattr(ops, "M3_ACT_" + name.upper())
    one = torch.ones((1, n), dtype=IO[io], device="cuda")
    x, W = one[:, :8].contiguous(), torch.ones((2 * n, 8), dtype=IO[io], device="cuda")
    h = z.double().cpu().numpy()
    f, df = exact(h, name)
    tol = bound(h, name, io)
    off = lambda got, ref: np.max(np.abs(got.double().cpu().numpy() - ref) / np.abs(ref) / tol)
    lin = ops.linear_bwd(x, W[:n], one, z.view(1, n), act=code, want_dx=False, want_dW=False)["dbias"]
    # gated, with u = 1: dP = [act'(g), act(g)]
    pre = torch.cat([z, torch.ones_like(z)]).view(1, 2 * n)
    gat = ops.gated_ffn_bwd(x, W, one, pre, act=code, want_dx=False, want_dW=False)["dbias"]
    worst = {"act' (linear)": off(lin, df), "act' (gated)": off(gat[:n], df), "act": off(gat[n:], f)}
    print(io, name, worst, flush=True)
    assert max(worst.values()) <= 1, worst


@pytest.mark.parametrize("io,name,far", TAILS)
def test_tails_in_the_forward(ops, io, name, far):
    # a product with the identity: pre is z, y is act(z) rounded once to the io type
    z = torch.linspace(5, far, 128).to(IO[io])
    n = z.numel()
    for rows in (2, 300):  # the few-row kernel, a tiled one
        x = torch.where(torch.arange(rows)[:, None] % 2 == 0, z, -z).to(IO[io]).cuda()
        W = torch.eye(n, dtype=IO[io], device="cuda")
        y, _ = ops.linear_fwd(x, W, act=getattr(ops, "M3_ACT_" + name.upper()))
        h = x.double().cpu().numpy()
        f, _ = exact(h.ravel(), name)
        tol = bound(h.ravel(), name, io) + (2.0 ** -8 if io == "bf16" else U)
        err = np.abs(y.double().cpu().numpy().ravel() - f) / np.abs(f) / tol
        print(io, name, rows, err.max(), flush=True)
        assert err.max() <= 1


def test_ends_of_the_activations(ops):
    # infinities and NaN: flat ends give 0 and 1, a NaN stays one
    inf, nan = float("inf"), float("nan")
    for io in ("bf16", "f32"):
        z = torch.tensor([[inf, -inf, nan, 200.0, -200.0, 0.0, 1e30, -1e30]], dtype=IO[io], device="cuda")
        one = torch.ones_like(z)
        W = torch.ones((8, 8), dtype=IO[io], device="cuda")
        d = lambda name: ops.linear_bwd(one, W, one, z, act=getattr(ops, "M3_ACT_" + name.upper()), want_dx=False,
                                        want_dW=False)["dbias"].tolist()
        got = d("sigmoid")
        assert got[:2] == [0.0, 0.0] and math.isnan(got[2]) and got[3:] == [0.0, 0.0, 0.25, 0.0, 0.0]
        for name in ("silu", "gelu", "gelu_tanh"):
            got = d(name)
            assert math.isnan(got[2]) and got[3] == 1.0 and got[4] == 0.0 and abs(got[5] - 0.5) < 1e-6
            assert got[6] == 1.0 and got[7] == 0.0
        got = d("relu")
        assert got[:2] == [1.0, 0.0] and math.isnan(got[2]) and got[3:] == [1.0, 0.0, 0.0, 1.0, 0.0]
