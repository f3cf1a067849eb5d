"""Parity of the residual block's operators with their fp64 oracle
(oracle/block.py, pinned in tests/test_oracle_block_pins.py).  Needs an MI355X.

Every output entry is held to the oracle's bound for it: one rounding of the
output (2^-8 of it covers bf16's half unit of 2^-9 and its neighbour's), one of
dP where the products take it as bf16, and a unit of 2^-23 per fp32 operation.
"""
import numpy as np
import pytest

from oracle import block

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -23
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print(*a, flush=True)


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from state_space_sequence_03_amd import ops as o
    o.lib()
    return o


def unit(io):
    return U_BF16 if io == "bf16" else U_F32


def host(t):
    return t.detach().double().cpu().numpy()


def draw(rng, shape, io, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda().to(IO[io])


def strided(t, pad, off):
    """The same values as a column slice of a wider matrix of NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, off:off + t.shape[1]] = t
    return wide, wide[:, off:off + t.shape[1]]


def within(name, got, ref, bound):
    got = host(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} entries off, first {i}: {got[i]} against {ref[i]}, "
                             f"bound {np.broadcast_to(bound, ref.shape)[i]}")


# ---------------------------------------------------------------------------
# layer norm: one wave per row (all register tiers), one block per row, rows
# re-read; odd widths, one column, one row
# ---------------------------------------------------------------------------
NORM = [(1, 1), (5, 3), (64, 64), (3, 511), (130, 512), (7, 1021), (33, 1024), (9, 2048), (10, 2050), (5, 4096),
        (3, 4100), (4, 8192), (3, 9001), (2, 20000)]


@pytest.mark.parametrize("rows,D", NORM)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_layer_norm(ops, io, rows, D):
    say(f"layer norm {io} {rows} x {D}")
    r = np.random.default_rng(D + rows)
    x = draw(r, (rows, D), io) * 2 + 0.5
    gain, bias = draw(r, D, "f32"), draw(r, D, "f32")
    u = unit(io)
    for g, b, eps in ((gain, bias, 1e-5), (None, None, 0.25)):
        y, mean, rstd = ops.layer_norm_fwd(x, g, b, eps, want_stats=True)
        hg, hb = (None if t is None else host(t) for t in (g, b))
        ref = block.layer_norm(host(x), hg, hb, eps)
        for name, t, want, bound in zip(("y", "mean", "rstd"), (y, mean, rstd), ref,
                                        block.layer_norm_bound(host(x), hg, hb, eps, u)):
            within(name, t, want, bound)
    dy, skip = draw(r, (rows, D), io), draw(r, (rows, D), io)
    hm, hr = host(mean), host(rstd)
    for g, sk in ((gain, skip), (None, None)):
        out = ops.layer_norm_bwd(x, mean, rstd, dy, g, sk)
        hg, hs = (None if t is None else host(t) for t in (g, sk))
        ref = block.layer_norm_bwd(host(x), hg, hm, hr, host(dy), hs)
        for name, want, bound in zip(("dx", "dgain", "dbias"), ref,
                                     block.layer_norm_bwd_bound(host(x), hg, hm, hr, host(dy), hs, u)):
            within(name, out[name], want, bound)
    # any subset of the outputs, the same values
    one = ops.layer_norm_bwd(x, mean, rstd, dy, None, want_dx=False, want_dbias=False)
    assert set(one) == {"dgain"} and torch.equal(one["dgain"], out["dgain"])
    two = ops.layer_norm_bwd(x, mean, rstd, dy, None, want_dgain=False, want_dbias=False)
    assert set(two) == {"dx"} and torch.equal(two["dx"], out["dx"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_layer_norm_many_rows(ops, io):
    # more rows than the backward has blocks: every block walks several, the last ones ragged
    r = np.random.default_rng(5)
    rows, D = 5003, 70
    x, dy = draw(r, (rows, D), io), draw(r, (rows, D), io)
    gain = draw(r, D, "f32")
    _, mean, rstd = ops.layer_norm_fwd(x, gain, want_stats=True)
    out = ops.layer_norm_bwd(x, mean, rstd, dy, gain)
    a = (host(x), host(gain), host(mean), host(rstd), host(dy), None)
    for name, want, bound in zip(("dx", "dgain", "dbias"), block.layer_norm_bwd(*a),
                                 block.layer_norm_bwd_bound(*a, unit(io))):
        within(name, out[name], want, bound)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D,pad,off", [(64, 64, 0), (64, 8, 8), (100, 3, 1), (2048, 24, 5), (4100, 11, 2)])
def test_layer_norm_strides(ops, io, D, pad, off):
    r = np.random.default_rng(D)
    x, dy, skip = (draw(r, (6, D), io) for _ in range(3))
    gain = draw(r, D, "f32")
    _, sx = strided(x, pad, off)
    _, sdy = strided(dy, pad + 1, off)
    wy, sy = strided(x, pad + 2, off)
    wsk, ssk = strided(skip, pad, off)
    y, mean, rstd = ops.layer_norm_fwd(x, gain, want_stats=True)
    ops.layer_norm_fwd(sx, gain, y=sy)
    assert torch.equal(sy, y)
    assert int(torch.isnan(wy).sum()) == 6 * (pad + 2)  # nothing written beside the rows
    ref = ops.layer_norm_bwd(x, mean, rstd, dy, gain, skip)
    out = ops.layer_norm_bwd(sx, mean, rstd, sdy, gain, ssk, dx=ssk)  # dx over dskip
    assert torch.equal(ssk, ref["dx"]) and torch.equal(out["dgain"], ref["dgain"])
    assert int(torch.isnan(wsk).sum()) == 6 * pad


def test_layer_norm_bad_rows_stay_alone(ops):
    # NaN, infinity and a constant row (eps = 0: 0/0) touch their own rows only
    r = np.random.default_rng(9)
    for io in ("bf16", "f32"):
        x = draw(r, (40, 200), io)
        good, _, _ = ops.layer_norm_fwd(x, eps=0.0)
        x[3, 7], x[11, 0], x[20] = float("nan"), float("inf"), 2.0
        y, _, _ = ops.layer_norm_fwd(x, eps=0.0)
        keep = [i for i in range(40) if i not in (3, 11, 20)]
        assert torch.equal(y[keep], good[keep])
        assert torch.isnan(y[[3, 11, 20]].float()).any(1).all()
        bias = draw(r, 200, "f32")
        y, _, rstd = ops.layer_norm_fwd(x, None, bias, 1e-5, want_stats=True)
        assert torch.equal(y[20], bias.to(IO[io])) and torch.isfinite(rstd[20])


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
# rows, d_in, d_out: single tokens, ragged tiles, odd widths, one column
SHAPES = [(1, 64, 64), (1, 1000, 130), (2, 17, 3), (16, 512, 96), (17, 64, 200), (33, 100, 1), (64, 128, 256),
          (65, 1, 65), (100, 333, 77), (128, 320, 128), (257, 192, 264), (300, 1031, 511), (520, 72, 520)]


def product_inputs(rng, io, M, K, N, is_gated):
    n = 2 * N if is_gated else N
    return (draw(rng, (M, K), io), draw(rng, (n, K), io, K ** -0.5), draw(rng, n, "f32"), draw(rng, (M, N), io))


def check_fwd(ops, io, name, x, W, bias, res, is_gated):
    code = getattr(ops, "M3_ACT_" + name.upper())
    hb, hr = (None if t is None else host(t) for t in (bias, res))
    if is_gated:
        y, pre = ops.gated_ffn_fwd(x, W, bias, act=code, want_pre=True)
        y2, none = ops.gated_ffn_fwd(x, W, bias, act=code)
        ref, bounds = block.gated(host(x), host(W), hb, name), block.gated_bound(host(x), host(W), hb, name, unit(io))
    else:
        y, pre = ops.linear_fwd(x, W, bias, res, act=code, want_pre=True)
        y2, none = ops.linear_fwd(x, W, bias, res, act=code)
        ref = block.linear(host(x), host(W), hb, hr, name)
        bounds = block.linear_bound(host(x), host(W), hb, hr, name, unit(io))
    within("y", y, ref[0], bounds[0])
    within("pre", pre, ref[1], bounds[1])
    assert none is None and torch.equal(y, y2)
    return pre


def check_bwd(ops, io, name, x, W, dy, pre, is_gated):
    code = getattr(ops, "M3_ACT_" + name.upper())
    call = ops.gated_ffn_bwd if is_gated else ops.linear_bwd
    out = call(x, W, dy, pre, act=code)
    hp, hd = None if pre is None else host(pre), host(dy)
    dp = block.dp_gated(hp, hd, name) if is_gated else block.dp_linear(hp, hd, name)
    u_dp = unit(io) if is_gated or name != "none" else 0.0
    bounds = block.products_bound(dp, block.dp_eval(hp, hd, name, is_gated), host(x), host(W), unit(io), u_dp)
    for key, want, bound in zip(("dx", "dW", "dbias"), block.products(dp, host(x), host(W)), bounds):
        within(key, out[key], want, bound)
    for key in ("dx", "dW", "dbias"):
        wants = {f"want_{k}": k == key for k in ("dx", "dW", "dbias")}
        one = call(x, W, dy, pre, act=code, **wants)
        assert set(one) == {key} and torch.equal(one[key], out[key])


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("is_gated", [False, True], ids=["linear", "gated"])
def test_products(ops, is_gated, io, M, K, N):
    r = np.random.default_rng(M * 7 + K * 3 + N)
    name = block.ACTS[(M + K + N) % 6]
    say(f"{'gated' if is_gated else 'linear'} {io} {M} x {K} x {N} {name}")
    x, W, bias, dy = product_inputs(r, io, M, K, N, is_gated)
    res = None if is_gated else draw(r, (M, N), io)
    pre = check_fwd(ops, io, name, x, W, bias, res, is_gated)
    check_bwd(ops, io, name, x, W, dy, pre, is_gated)


@pytest.mark.parametrize("name", block.ACTS)
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(5, 64, 48), (140, 128, 136)])
def test_every_activation(ops, io, name, M, K, N):
    r = np.random.default_rng(21)
    for is_gated in (False, True):
        x, W, bias, dy = product_inputs(r, io, M, K, N, is_gated)
        x = x * 3  # reach the activations' flat ends
        for b in (bias, None):
            pre = check_fwd(ops, io, name, x, W, b, None, is_gated)
        check_bwd(ops, io, name, x, W, dy, pre, is_gated)


# larger products: every tile form, k split over blocks, many rows with few columns
BIG = [(2100, 512, 1100, "silu"), (8200, 256, 64, "none"), (700, 2048, 1408, "gelu"), (48, 4096, 512, "gelu_tanh"),
       (200, 5000, 96, "relu"), (12000, 64, 96, "sigmoid")]


@pytest.mark.parametrize("M,K,N,name", BIG)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_larger_products(ops, io, M, K, N, name):
    r = np.random.default_rng(M + N)
    for is_gated in (False, True):
        say(f"{'gated' if is_gated else 'linear'} {io} {M} x {K} x {N} {name}")
        x, W, bias, dy = product_inputs(r, io, M, K, N, is_gated)
        res = None if is_gated else draw(r, (M, N), io)
        pre = check_fwd(ops, io, name, x, W, bias, res, is_gated)
        check_bwd(ops, io, name, x, W, dy, pre, is_gated)


# the widest tiles: more of them than CUs, so that some are whole and the last
# ones split over k, with ragged edges (M, N) or none (4096), K short, odd or
# off the tile's stages
WIDE = [(4100, 520, 4000, "silu"), (4096, 200, 4352, "gelu"), (8200, 65, 2304, "none"), (4097, 1031, 4103, "relu")]


@pytest.mark.parametrize("M,K,N,name", WIDE)
def test_wide_tiles(ops, M, K, N, name):
    r = np.random.default_rng(M + K)
    for is_gated in (False, True):
        n = N // 2 if is_gated else N
        say(f"{'gated' if is_gated else 'linear'} {M} x {K} x {n} {name}")
        x, W, bias, dy = product_inputs(r, "bf16", M, K, n, is_gated)
        res = None if is_gated else draw(r, (M, n), "bf16")
        pre = check_fwd(ops, "bf16", name, x, W, bias, res, is_gated)
        check_fwd(ops, "bf16", name, x, W, None, None, is_gated)
        check_bwd(ops, "bf16", name, x, W, dy, pre, is_gated)


def test_wide_tiles_f32(ops):
    r = np.random.default_rng(77)
    for is_gated in (False, True):
        n = 2000 if is_gated else 4000
        x, W, bias, dy = product_inputs(r, "f32", 4100, 132, n, is_gated)
        pre = check_fwd(ops, "f32", "silu", x, W, bias, None, is_gated)
        check_bwd(ops, "f32", "silu", x, W, dy, pre, is_gated)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(5, 64, 48), (70, 64, 72), (300, 512, 256)])
def test_pointers_off_16_bytes(ops, io, M, K, N):
    # rows of whole 16 bytes that start off them: every operand a view one element into its buffer
    r = np.random.default_rng(M + K + N)

    def off(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)

    for is_gated in (False, True):
        x, W, bias, dy = product_inputs(r, io, M, K, N, is_gated)
        pre = check_fwd(ops, io, "silu", off(x), off(W), off(bias), None, is_gated)
        check_bwd(ops, io, "silu", off(x), off(W), off(dy), off(pre), is_gated)
        if not is_gated:
            check_bwd(ops, io, "none", x, W, off(dy), None, False)


def test_graph_replays(ops):
    # a block's forward and backward captured once; every replay equals the eager call
    r = np.random.default_rng(55)
    x, W, bias, dy = product_inputs(r, "bf16", 1000, 264, 520, True)
    gain = draw(r, 264, "f32")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def block_step():
        n, mean, rstd = ops.layer_norm_fwd(x, gain, want_stats=True)
        h, pre = ops.gated_ffn_fwd(n, W, bias, want_pre=True, workspace=ws)
        g = ops.gated_ffn_bwd(n, W, dy, pre, workspace=ws)
        b = ops.layer_norm_bwd(x, mean, rstd, g["dx"], gain, workspace=ws)
        return [h, g["dW"], g["dbias"], b["dx"], b["dgain"], b["dbias"]]

    block_step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block_step()
    for k in range(4):
        x.copy_(draw(r, (1000, 264), "bf16"))
        want = [t.clone() for t in block_step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N,pad,off", [(70, 64, 72, 64, 0), (70, 64, 72, 8, 8), (130, 100, 70, 3, 1),
                                           (3, 256, 128, 5, 3), (300, 512, 256, 16, 8)])
def test_product_strides(ops, io, M, K, N, pad, off):
    r = np.random.default_rng(M)
    for is_gated in (False, True):
        x, W, bias, dy = product_inputs(r, io, M, K, N, is_gated)
        _, sx = strided(x, pad, off)
        _, sdy = strided(dy, pad + 1, off)
        wy, sy = strided(dy, pad + 2, off)
        if is_gated:
            y, pre = ops.gated_ffn_fwd(x, W, bias, want_pre=True)
            ops.gated_ffn_fwd(sx, W, bias, h=sy)
            ref, out = ops.gated_ffn_bwd(x, W, dy, pre), ops.gated_ffn_bwd(sx, W, sdy, pre)
        else:
            res = draw(r, (M, N), io)
            _, sres = strided(res, pad + 3, off)
            y, _ = ops.linear_fwd(x, W, bias, res)
            ops.linear_fwd(sx, W, bias, sres, y=sy)
            ref, out = ops.linear_bwd(x, W, dy), ops.linear_bwd(sx, W, sdy)
        # the same sums in another order where a layout takes another kernel
        tol = 2 * unit(io) if io == "bf16" else 1e-4
        assert torch.allclose(sy.float(), y.float(), rtol=tol, atol=tol * float(y.float().abs().max()))
        assert int(torch.isnan(wy).sum()) == M * (pad + 2)
        for k in ref:
            a, b = out[k].float(), ref[k].float()
            assert torch.allclose(a, b, rtol=tol, atol=tol * float(b.abs().max())), k


def test_bad_values_stay_in_their_rows_and_columns(ops):
    # a NaN or infinity in one row of x reaches that row of y only; in one row
    # of W that column only (tiles are padded with zeros, never with neighbours)
    r = np.random.default_rng(31)
    for io in ("bf16", "f32"):
        for M, K, N in ((70, 100, 90), (5, 72, 40), (300, 192, 136)):
            x, W, bias, _ = product_inputs(r, io, M, K, N, False)
            good, _ = ops.linear_fwd(x, W, bias, act=ops.M3_ACT_RELU)
            x2, W2 = x.clone(), W.clone()
            x2[M - 1, K - 1], W2[N - 1, K - 1] = float("nan"), float("inf")
            bad, _ = ops.linear_fwd(x2, W2, bias, act=ops.M3_ACT_RELU)
            assert torch.equal(bad[:-1, :-1], good[:-1, :-1]), (io, M, K, N)
            assert torch.isnan(bad[-1].float()).all()
            assert not torch.isfinite(bad[:-1, -1].float()).all()


@pytest.mark.parametrize("M,K,N", [(70, 64, 90), (2100, 512, 260), (3, 2048, 512)])
def test_repeats_are_bitwise_equal_and_stay_inside(ops, M, K, N):
    # outputs and workspaces between guard bytes, a side stream, no dependence on timing
    r = np.random.default_rng(41)
    for io in ("bf16", "f32"):
        x, W, bias, dy = product_inputs(r, io, M, K, N, True)
        side = torch.cuda.Stream()

        def guarded(shape, dtype):
            n = int(np.prod(shape)) * dtype.itemsize
            raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
            return raw, raw[256:256 + n].view(dtype).view(shape)

        got = []
        for _ in range(2):
            raws = []

            def out(shape, dtype=IO[io]):
                raw, t = guarded(shape, dtype)
                raws.append(raw)
                return t

            h, pre, dx, dW, db = (out((M, N)), out((M, 2 * N)), out((M, K)), out((2 * N, K)),
                                  out((2 * N,), torch.float32))
            dims = ops.LinearDims(M, K, N, 0, 0, 0, ops._io_code(x), ops.M3_ACT_SILU, 0, 0)
            wf, wb = (out((max(16, n),), torch.uint8) for n in (ops.gated_ffn_fwd_workspace_size(dims),
                                                               ops.gated_ffn_bwd_workspace_size(dims)))
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                ops.gated_ffn_fwd(x, W, bias, h=h, pre=pre, workspace=wf)
                ops.gated_ffn_bwd(x, W, dy, pre, dx=dx, dW=dW, dbias=db, workspace=wb)
            torch.cuda.synchronize()
            for raw in raws:
                assert int((raw[:256] != 0xA5).sum()) == 0 and int((raw[-256:] != 0xA5).sum()) == 0
            got.append([t.clone() for t in (h, pre, dx, dW, db)])
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_no_rows(ops):
    for io in ("bf16", "f32"):
        x = torch.empty((0, 40), dtype=IO[io], device="cuda")
        W = torch.ones((12, 40), dtype=IO[io], device="cuda")
        assert ops.linear_fwd(x, W)[0].shape == (0, 12)
        assert ops.gated_ffn_fwd(x, W)[0].shape == (0, 6)
        full = lambda *s, dt=IO[io]: torch.full(s, 7.0, dtype=dt, device="cuda")
        g = ops.linear_bwd(x, W, x[:, :12], dW=full(12, 40), dbias=full(12, dt=torch.float32))
        assert not g["dW"].any() and not g["dbias"].any() and g["dx"].shape == (0, 40)
        g = ops.gated_ffn_bwd(x, W, x[:, :6], x[:, :12].contiguous(), dW=full(12, 40))
        assert not g["dW"].any() and not g["dbias"].any()
        y, mean, rstd = ops.layer_norm_fwd(x, want_stats=True)
        assert y.shape == (0, 40) and mean.shape == (0,)
        g = ops.layer_norm_bwd(x, mean, rstd, x, dgain=full(40, dt=torch.float32))
        assert not g["dgain"].any() and not g["dbias"].any()


def test_offsets_past_32_bits(ops):
    # 1.1 M rows of 2048 bf16 are 4.5 GB: byte offsets and element counts pass 2^32 and 2^31
    M, K, N = 1_100_003, 2048, 24
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for i in range(0, M, 1 << 17):
        x[i:i + (1 << 17)] = torch.randn((min(1 << 17, M - i), K), device="cuda", generator=g).to(torch.bfloat16)
    W = (torch.randn((N, K), device="cuda", generator=g) * K ** -0.5).to(torch.bfloat16)
    dy = torch.randn((M, N), device="cuda", generator=g).to(torch.bfloat16)
    say("rows past 32 bits: forward")
    pick = torch.tensor([0, 1, M // 2, 1_048_575, 1_048_576, M - 2, M - 1], device="cuda")
    y, _ = ops.linear_fwd(x, W)
    ref = block.linear(host(x[pick]), host(W), None, None, "none")[0]
    within("y", y[pick], ref, block.linear_bound(host(x[pick]), host(W), None, None, "none", U_BF16)[0])
    n, mean, rstd = ops.layer_norm_fwd(x, want_stats=True)
    ref = block.layer_norm(host(x[pick]), None, None, 1e-5)[0]
    within("norm", n[pick], ref, block.layer_norm_bound(host(x[pick]), None, None, 1e-5, U_BF16)[0])
    del n
    say("rows past 32 bits: backward")
    out = ops.linear_bwd(x, W, dy)
    within("dx", out["dx"][pick], host(dy[pick]) @ host(W),
           block.products_bound(host(dy[pick]), 0 * host(dy[pick]), host(x[pick]), host(W), U_BF16, 0.0)[0])
    # dW in fp64 on the device, a slice of rows at a time (fp64 products only)
    dW, mag = torch.zeros((N, K), dtype=torch.float64, device="cuda"), 0.0
    for i in range(0, M, 1 << 16):
        a, b = dy[i:i + (1 << 16)].double(), x[i:i + (1 << 16)].double()
        dW += a.t() @ b
        mag = mag + a.abs().t() @ b.abs()
    # fp32 sums of M terms whose signs are random: a few square roots of M units of the sum of squares' root
    bound = U_BF16 * dW.abs() + 64 * U_F32 * mag
    assert bool(((out["dW"].double() - dW).abs() <= bound).all())
