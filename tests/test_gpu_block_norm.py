"""Layer norm's backward of rows that are re-read (wider than a block holds) and
of many rows, where the column sums go through partial rows.  Needs an MI355X.

Every entry is held to the oracle's bound (oracle/block.py).
"""
import numpy as np
import pytest

from oracle import block

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
U_OUT = {"bf16": 2.0 ** -8, "f32": 2.0 ** -23}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from state_space_sequence_03_amd import ops as o
    o.lib()
    return o


# one slab of rows, several, more rows than slabs, one slab for many rows (the widest)
@pytest.mark.parametrize("rows,D", [(9, 8193), (40, 9001), (300, 20000), (1500, 8200), (33, 300_001), (12, 1 << 20),
                                    (1100, 2049), (2500, 1021), (700, 4096)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_norm_backward(ops, io, rows, D):
    print("norm backward", io, rows, D, flush=True)
    r = np.random.default_rng(rows + D)
    draw = lambda *s: torch.from_numpy(r.standard_normal(s, dtype=np.float32)).cuda()
    x, dy, skip = (draw(rows, D).to(IO[io]) for _ in range(3))
    gain = draw(D)
    _, mean, rstd = ops.layer_norm_fwd(x, gain, want_stats=True)
    out = ops.layer_norm_bwd(x, mean, rstd, dy, gain, skip)
    host = lambda t: t.double().cpu().numpy()
    a = [host(t) for t in (x, gain, mean, rstd, dy, skip)]
    for name, want, bound in zip(("dx", "dgain", "dbias"), block.layer_norm_bwd(*a),
                                 block.layer_norm_bwd_bound(*a, U_OUT[io])):
        got = host(out[name])
        assert got.shape == want.shape
        off = ~(np.abs(got - want) <= bound)
        assert not off.any(), (name, int(off.sum()), np.argwhere(off)[0])
    again = ops.layer_norm_bwd(x, mean, rstd, dy, gain, skip)
    assert all(torch.equal(again[k], out[k]) for k in out)
