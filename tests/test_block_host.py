"""More host-side checks of the residual block's entry points (no GPU, nothing
is launched): calls that ask for nothing, and the arithmetic of workspaces and
plans at the limits of what is accepted.  tests/test_block_sanitized.py runs
them again under sanitizers."""
import pytest

from test_block_abi import BWD, FAKE, L, call, lin, norm  # noqa: F401  (L is a fixture)

NOTHING = dict(dx=None, dW=None, dbias=None)


@pytest.mark.parametrize("fn", ["linear_bwd", "gated_ffn_bwd"])
def test_no_gradient_asked_for(L, fn):
    # nothing to do: no workspace is needed, and none is touched
    for dims in (lin(L), lin(L, rows=500, d_in=1001, d_out=77), lin(L, rows=0)):
        assert call(L, fn, BWD, dims, ws=None, ws_bytes=0, **NOTHING) == L.M3_OK
    # ... but the arguments are still checked
    assert call(L, fn, BWD, lin(L, act=6), ws=None, ws_bytes=0, **NOTHING) == L.M3_ERR_UNSUPPORTED
    assert call(L, fn, BWD, lin(L), x=FAKE + 1, ws=None, ws_bytes=0, **NOTHING) == L.M3_ERR_ALIGN


def test_largest_sizes(L):
    # every size query at the documented limits: sums that pass 32 bits
    rows, wide = (1 << 24) - 1, 1 << 20
    need = L.layer_norm_bwd_workspace_size(norm(L, rows=rows, width=wide))
    assert need % (8 * wide) == 0 and need > 0
    for flags in (0, L.M3_FLAG_UNALIGNED):
        for io in (L.M3_BF16, L.M3_F32):
            for kw in (dict(rows=rows, d_in=wide, d_out=1), dict(rows=rows, d_in=64, d_out=64),
                       dict(rows=65, d_in=wide, d_out=1 << 19), dict(rows=1, d_in=wide, d_out=1 << 19)):
                d = lin(L, io_dtype=io, flags=flags, **kw)
                copies = 0
                if flags:  # x and W are copied
                    copies = (kw["rows"] * kw["d_in"] if kw["rows"] > 64 else 0) * (2 if io == L.M3_BF16 else 4)
                for fn in ("linear", "gated_ffn"):
                    assert getattr(L, fn + "_fwd_workspace_size")(d) >= copies
                    getattr(L, fn + "_bwd_workspace_size")(d)


@pytest.mark.parametrize("io", ["M3_BF16", "M3_F32"])
def test_norm_workspace_is_bounded(L, io):
    # partial column sums: 1024 rows of the widest row that a block holds, and 16
    # MB where rows are wider than that
    held = 8192 if io == "M3_BF16" else 4096
    for rows in (1, 9, 300, 2048, 100_000, (1 << 24) - 1):
        for width in (1, 64, 1021, 2048, held, held + 1, 9001, 20000, 65536, 1 << 20):
            need = L.layer_norm_bwd_workspace_size(norm(L, rows=rows, width=width, io_dtype=getattr(L, io)))
            assert need > 0 and need % (8 * width) == 0
            assert rows > 8 or need == 8 * width
            assert need <= (1024 * 8 * held if width <= held else 1 << 24)
