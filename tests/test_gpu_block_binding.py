"""What the residual block's calls allocate themselves: with stream= it stays
theirs until their kernels are done; an output has its operand's shape.  Needs
an MI355X."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from state_space_sequence_03_amd import ops as o
    o.lib()
    return o


def tensors(out):
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_workspaces_outlive_their_call(ops, dtype):
    # the given stream is held up, so that every kernel runs long after its call
    # returned and dropped its workspace; meanwhile the current stream takes and
    # overwrites all the memory it can get of those sizes
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(dtype)
    M, K, F = 300, 333, 129  # odd rows: copies of x and W, dP, split parts and column sums in the workspace
    x, W, V, dh, dy = rand(M, K), rand(2 * F, K), rand(F, K), rand(M, F), rand(M, K)
    gain = torch.randn(K, device="cuda", generator=g)
    _, mean, rstd = ops.layer_norm_fwd(x, gain, want_stats=True)
    _, pre = ops.gated_ffn_fwd(x, W, want_pre=True)
    calls = [lambda **k: ops.layer_norm_bwd(x, mean, rstd, dy, gain, **k),
             lambda **k: ops.linear_fwd(x, V, act=ops.M3_ACT_GELU, want_pre=True, **k),
             lambda **k: ops.linear_bwd(x, V, dh, **k),
             lambda **k: ops.gated_ffn_fwd(x, W, want_pre=True, **k),
             lambda **k: ops.gated_ffn_bwd(x, W, dh, pre, **k)]
    side = torch.cuda.Stream()
    for i, call in enumerate(calls):
        print("call", i, flush=True)
        want = [t.clone() for t in tensors(call())]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about ten milliseconds
        got = tensors(call(stream=side))
        fill = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
                for n in (1 << 10, 1 << 12, 1 << 14, 1 << 16, 1 << 18, 400_000, 1 << 19, 900_000, 1 << 20, 1 << 21) * 3]
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        del fill


def test_norm_of_three_dimensions_with_a_strided_skip(ops):
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g)
    x, dy, wide = rand(3, 5, 64), rand(3, 5, 64), rand(15, 100)
    skip = wide[:, 7:71]
    _, mean, rstd = ops.layer_norm_fwd(x, want_stats=True)
    want = ops.layer_norm_bwd(x, mean, rstd, dy, dskip=skip.contiguous())
    got = ops.layer_norm_bwd(x, mean, rstd, dy, dskip=skip)
    assert got["dx"].shape == x.shape and torch.equal(got["dx"], want["dx"])
    assert torch.equal(got["dgain"], want["dgain"])
