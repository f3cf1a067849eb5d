"""The residual block's operators with infinities and NaN in one place of an
operand.  Needs an MI355X."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from state_space_sequence_03_amd import ops as o
    o.lib()
    return o


# a form of each tile, with whole and with split tiles, odd widths that are copied first
PLACES = [(1, 64, 64), (5, 72, 40), (70, 100, 90), (300, 192, 136), (129, 333, 257), (2100, 512, 260), (700, 2048, 1408),
          (4100, 520, 2300)]


def same_but(got, want, rows=None, cols=None):
    """Equal outside the given row and column; not finite inside them."""
    keep = torch.ones_like(want, dtype=torch.bool)
    if rows is not None:
        keep[rows] = False
    if cols is not None:
        keep[:, cols] = False
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[~keep].float()).any()


@pytest.mark.parametrize("M,K,N", PLACES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_bad_values_stay_in_their_place_in_the_backward(ops, gated, io, M, K, N):
    # dx = dP W, dW = dP^T x: a bad entry of x reaches one column of dW, one of
    # W one column of dx, one of dy its row of dx and its row(s) of dW and dbias
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K + N)
    rand = lambda *s: (torch.randn(s, device="cuda", generator=g) + 3).to(IO[io])  # away from 0: no inf * 0
    n = 2 * N if gated else N
    x, W, dy, pre = rand(M, K), rand(n, K), rand(M, N), rand(M, n)
    call = ops.gated_ffn_bwd if gated else ops.linear_bwd
    run = lambda x=x, W=W, dy=dy: call(x, W, dy, pre, act=ops.M3_ACT_SIGMOID)
    good = run()
    for bad in (float("nan"), float("inf")):
        for m, k, j in ((M - 1, K - 1, N - 1), (0, 0, 0), (M // 2, K // 3, N // 2)):
            print(io, gated, M, K, N, bad, (m, k, j), flush=True)
            t = x.clone()
            t[m, k] = bad
            out = run(x=t)
            assert torch.equal(out["dx"], good["dx"]) and torch.equal(out["dbias"], good["dbias"])
            same_but(out["dW"], good["dW"], cols=[k])
            t = W.clone()
            t[n - 1 - j, k] = bad
            out = run(W=t)
            assert torch.equal(out["dW"], good["dW"]) and torch.equal(out["dbias"], good["dbias"])
            same_but(out["dx"], good["dx"], cols=[k])
            t = dy.clone()
            t[m, j] = bad
            out = run(dy=t)
            same_but(out["dx"], good["dx"], rows=[m])
            mine = [j, N + j] if gated else [j]
            same_but(out["dW"], good["dW"], rows=mine)
            same_but(out["dbias"][:, None], good["dbias"][:, None], rows=mine)


@pytest.mark.parametrize("M,K,N", PLACES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
def test_bad_values_stay_in_their_place_in_the_forward(ops, gated, io, M, K, N):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K + N)
    rand = lambda *s: (torch.randn(s, device="cuda", generator=g) + 3).to(IO[io])
    n = 2 * N if gated else N
    x, W, bias = rand(M, K), rand(n, K), torch.randn(n, device="cuda", generator=g)
    call = ops.gated_ffn_fwd if gated else ops.linear_fwd
    run = lambda x=x, W=W, bias=bias: call(x, W, bias, act=ops.M3_ACT_NONE, want_pre=True)
    y, pre = run()
    for bad in (float("nan"), float("inf")):
        for m, k, j in ((M - 1, K - 1, n - 1), (0, 0, 0), (M // 2, K // 3, n // 2)):
            t = x.clone()
            t[m, k] = bad
            y2, pre2 = run(x=t)
            same_but(pre2, pre, rows=[m])
            same_but(y2, y, rows=[m])
            t = W.clone()
            t[j, k] = bad
            y2, pre2 = run(W=t)
            same_but(pre2, pre, cols=[j])
            same_but(y2, y, cols=[j % N])
            t = bias.clone()
            t[j] = bad
            y2, pre2 = run(bias=t)
            same_but(pre2, pre, cols=[j])
            same_but(y2, y, cols=[j % N])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(1, 1), (4, 64), (37, 300), (70, 1021), (40, 2048), (12, 5000), (9, 9001)])
def test_bad_values_in_the_norm_backward(ops, io, rows, D):
    # a bad entry of x or dy reaches its own row of dx and, in dgain and dbias,
    # its row's share of every column it enters
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + D)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(IO[io])
    x, dy, skip = rand(rows, D), rand(rows, D), rand(rows, D)
    _, mean, rstd = ops.layer_norm_fwd(x, want_stats=True)
    good = ops.layer_norm_bwd(x, mean, rstd, dy, None, skip)
    for m, k in ((rows - 1, D - 1), (0, 0), (rows // 2, D // 2)):
        for bad in (float("nan"), float("inf")):
            t = dy.clone()
            t[m, k] = bad
            out = ops.layer_norm_bwd(x, mean, rstd, t, None, skip)
            keep = torch.arange(rows, device="cuda") != m
            assert torch.equal(out["dx"][keep], good["dx"][keep])
            assert torch.isnan(out["dx"][m].float()).any()
            for key in ("dgain", "dbias"):  # that column only
                cols = torch.arange(D, device="cuda") != k
                assert torch.equal(out[key][cols], good[key][cols])
                assert D == 1 and key == "dgain" or not torch.isfinite(out[key][k])
            t = skip.clone()
            t[m, k] = bad
            out = ops.layer_norm_bwd(x, mean, rstd, dy, None, t)
            same = torch.ones_like(x, dtype=torch.bool)
            same[m, k] = False
            assert torch.equal(out["dx"][same], good["dx"][same]) and not torch.isfinite(out["dx"][m, k].float())
            assert torch.equal(out["dgain"], good["dgain"]) and torch.equal(out["dbias"], good["dbias"])
