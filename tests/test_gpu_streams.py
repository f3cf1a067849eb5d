"""Calls with stream=: what a call of the layer core allocates stays its own
until its kernels are done, and such calls can be captured.  Needs an MI355X."""
import pytest

from state_space_sequence_03_amd.inputs import prologue_torch, torch_inputs

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
    return [t for t in (out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,))
            if t is not None]


def core_calls(ops):
    b, L, H, P, N, R, D = 2, 700, 3, 64, 64, 4, 128
    d = torch_inputs(b, L, H, P, N, R, io="bf16", seed=5)
    s = [d[k] for k in ("x", "B", "C", "dt", "A", "lam", "theta")]
    dy, token = torch.randn_like(d["x"]), [t[:, 0].contiguous() for t in s]
    state = torch.randn((b, H, N, P), device="cuda")
    p = prologue_torch(b, L, H, N, R, D, seed=6)
    yield "chunked_fwd", lambda **k: ops.chunked_fwd(*s, segments=4, **k)
    yield "chunked_bwd", lambda **k: ops.chunked_bwd(*s, dy, **k)
    yield "rope_bc", lambda **k: ops.rope_bc(d["B"], d["C"], d["dt"], d["theta"], **k)
    yield "bc_prologue", lambda **k: ops.bc_prologue(p["u"], p["W"], p["dt"], p["theta"], H, R, N, **k)

    def decode(**k):
        with torch.cuda.stream(k.get("stream")):  # the state is the call's own, made where it runs
            h = state.clone()
        return ops.decode_step(h, *token, **k), h

    yield "decode_step", decode


def test_workspaces_outlive_their_call(ops):
    # the given stream is held up while the current one takes and overwrites
    # all the memory it can get
    side = torch.cuda.Stream()
    for name, call in core_calls(ops):
        print(name, flush=True)
        want = [t.clone() for t in tensors(call())]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about ten milliseconds
        got = tensors(call(stream=side))
        fill = [torch.full((1 << n,), 0xFF, dtype=torch.uint8, device="cuda") for n in range(10, 25)] * 2
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        del fill


def test_captured_with_a_stream(ops):
    # a branch of a graph on another stream, with stream=: every replay equals the eager call
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()
    x, W, dh = rand(300, 264), rand(2 * 130, 264), rand(300, 130)
    d = torch_inputs(1, 200, 2, 64, 64, 1, io="bf16", seed=9)
    core = [d[k] for k in ("x", "B", "C", "dt", "A", "lam", "theta")]
    branch = torch.cuda.Stream()

    def step(**k):
        h, pre = ops.gated_ffn_fwd(x, W, want_pre=True, **k)
        grad = ops.gated_ffn_bwd(x, W, dh, pre, **k)
        y, hf = ops.chunked_fwd(*core, **k)
        return [h, grad["dx"], grad["dW"], grad["dbias"], y, hf]

    step(stream=branch)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        branch.wait_stream(torch.cuda.current_stream())
        out = step(stream=branch)
        torch.cuda.current_stream().wait_stream(branch)
    for k in range(4):
        x.copy_(rand(300, 264))
        core[0].copy_(torch.randn_like(core[0]))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
