"""Every form of the products that the planner picks (the list, and the pin of
each size to its form, are in tests/test_block_plans.py), against the formula in
64 bits, entry by entry.  Needs an MI355X.

The bounds are the oracle's (oracle/block.py): a unit of 2^-23 per term of a
fp32 sum, the activation's evaluation, one rounding of each output.  The
products of the reference run in fp64 on the device.
"""
import math

import pytest

from oracle import block
from test_block_plans import ALL, IDS, form, plan  # noqa: F401  (plan is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
U_OUT = {"bf16": 2.0 ** -8, "f32": block.U32}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from state_space_sequence_03_amd import ops as o
    o.lib()
    return o


def act64(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return torch.sigmoid(z) if name == "sigmoid" else z


def within(name, got, ref, bound):
    assert got.shape == ref.shape
    off = ~((got.double() - ref).abs() <= bound)  # a NaN is off
    if off.any():
        i = tuple(int(v) for v in off.nonzero()[0])
        raise AssertionError(f"{name}: {int(off.sum())} of {off.numel()} entries off, first {i}: {float(got[i])} "
                             f"against {float(ref[i])}, bound {float(bound[i])}")


def check_fwd(io, name, x, W, bias, res, y, pre, gated):
    u, U = U_OUT[io], block.U32
    x, W = x.double(), W.double()
    z = x @ W.t()
    e = (x.shape[1] + 16) * U * (x.abs() @ W.abs().t())
    if bias is not None:
        z = z + bias
        e = e + U * (z.abs() + bias.abs())
    within("pre", pre, z, e * (1 + u) + u * z.abs() + 1e-30)
    F = W.shape[0] // 2 if gated else W.shape[0]
    g, eg = z[:, :F], e[:, :F]
    f = act64(g, name)
    ef = block.SLOPE * eg + (0 if name in ("none", "relu") else block.ACT_EVAL) * g.abs().clamp(min=1)
    if gated:
        v, ev = z[:, F:], e[:, F:]
        ef = ef * (v.abs() + ev) + f.abs() * ev
        f = f * v
    elif res is not None:
        f = f + res.double()
    within("y", y, f, (ef + 2 * U * f.abs()) * (1 + u) + u * f.abs() + 1e-30)


class Guarded:
    """Outputs between guard bytes."""

    def __init__(self):
        self.raw = []

    def __call__(self, shape, dtype):
        n = math.prod(shape) * dtype.itemsize
        raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        self.raw.append(raw)
        return raw[256:256 + n].view(dtype).view(shape)

    def check(self):
        for raw in self.raw:
            assert int((raw[:256] != 0xA5).sum()) == 0 and int((raw[-256:] != 0xA5).sum()) == 0


@pytest.mark.parametrize("case", ALL, ids=IDS)
def test_form(ops, plan, case):  # noqa: F811
    kind, io, M, K, N = case[:5]
    print("form", *case, flush=True)
    assert form(plan, *case[:5]) == case[5:]
    g = torch.Generator(device="cuda")
    g.manual_seed(M + 3 * K + 7 * N)
    rand = lambda *s, scale=1.0, dtype=IO[io]: (torch.randn(s, device="cuda", generator=g) * scale).to(dtype)
    u, U = U_OUT[io], block.U32
    out = Guarded()
    if kind in ("dx", "dW"):
        x, W, dy = rand(M, K), rand(N, K), rand(M, N)
        keep = out((M, K) if kind == "dx" else (N, K), IO[io])
        want = {"want_dx": kind == "dx", "want_dW": kind == "dW", "want_dbias": False}
        ops.linear_bwd(x, W, dy, **{kind: keep}, **want)
        a, b = (dy.double(), W.double()) if kind == "dx" else (dy.double().t(), x.double())
        ref, e = a @ b, (a.shape[1] + 16) * U * (a.abs() @ b.abs())
        within(kind, keep, ref, e * (1 + u) + u * ref.abs() + 1e-30)
        again = ops.linear_bwd(x, W, dy, **want)[kind]
        assert torch.equal(again, keep)
    else:
        gated = kind == "gated"
        n = 2 * N if gated else N
        x, W, bias = rand(M, K), rand(n, K, scale=K ** -0.5), rand(n, dtype=torch.float32)
        name = block.ACTS[(M + K + N) % 6]
        code = getattr(ops, "M3_ACT_" + name.upper())
        y, pre = out((M, N), IO[io]), out((M, n), IO[io])
        if gated:
            res = None
            ops.gated_ffn_fwd(x, W, bias, act=code, h=y, pre=pre)
            again = ops.gated_ffn_fwd(x, W, bias, act=code)[0]
        else:
            res = rand(M, N)
            ops.linear_fwd(x, W, bias, res, act=code, y=y, pre=pre)
            again = ops.linear_fwd(x, W, bias, res, act=code)[0]
        check_fwd(io, name, x, W, bias.double(), res, y, pre, gated)
        assert torch.equal(again, y)
        # the epilogue with nothing but the product
        if gated:
            y, pre = ops.gated_ffn_fwd(x, W, act=ops.M3_ACT_NONE, want_pre=True)
        else:
            y, pre = ops.linear_fwd(x, W, want_pre=True)
        check_fwd(io, "none", x, W, None, None, y, pre, gated)
    out.check()
