"""The binding on the host: where its allocations go, what the residual block's
calls refuse and the shapes they return.  No GPU and no launch: the library is a
stand-in that takes every call, and operands lie in host memory.
"""
import contextlib

import pytest

torch = pytest.importorskip("torch")
from torch.utils._python_dispatch import TorchDispatchMode  # noqa: E402

from state_space_sequence_03_amd import ops  # noqa: E402


class Library:
    """Every entry point answers 0 (ok), every workspace query 4096."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda dims: 4096
        return lambda *a: self.calls.append((name, a)) or 0


class Stream:
    device = torch.device("cpu")
    cuda_stream = 0x51DE


@pytest.fixture
def fake(monkeypatch):
    """ops on the stand-in; .inside: the stream a with block has made current."""
    library = Library()
    library.inside, library.recorded = None, []

    @contextlib.contextmanager
    def stream(s):
        old, library.inside = library.inside, s
        yield
        library.inside = old

    class Current:
        cuda_stream = property(lambda self: 0 if library.inside is None else library.inside.cuda_stream)

    monkeypatch.setattr(ops, "lib", lambda: library)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Current())
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: library.recorded.append(t), raising=False)
    return library


def block_calls():
    """Each entry point on small operands: its name, the call, the outputs it makes itself."""
    x, W, V = torch.ones(4, 16), torch.ones(6, 16), torch.ones(6)
    m, g = torch.ones(4), torch.ones(16)
    yield "layer_norm_fwd", lambda **k: ops.layer_norm_fwd(x, g, want_stats=True, **k), 3
    yield "layer_norm_bwd", lambda **k: ops.layer_norm_bwd(x, m, m, x, g, **k), 3
    yield "linear_fwd", lambda **k: ops.linear_fwd(x, W, V, act=ops.M3_ACT_SILU, want_pre=True, **k), 2
    yield "linear_bwd", lambda **k: ops.linear_bwd(x, W, torch.ones(4, 6), **k), 3
    yield "gated_ffn_fwd", lambda **k: ops.gated_ffn_fwd(x, W, V, want_pre=True, **k), 2
    yield "gated_ffn_bwd", lambda **k: ops.gated_ffn_bwd(x, W, torch.ones(4, 3), torch.ones(4, 6), **k), 3


BLOCK = [name for name, _, _ in block_calls()]


def core_calls():
    """The same for the layer core's entry points that allocate."""
    b, L, H, R, P, N = 1, 3, 2, 1, 16, 16
    x, B, s, th = torch.ones(b, L, H, R, P), torch.ones(b, L, H, R, N), torch.ones(b, L, H), torch.ones(b, L, H, N // 2)
    h, token = torch.ones(b, H, N, P), [t[:, 0].contiguous() for t in (x, B, B, s, s, s, th)]
    u, W = torch.ones(b, L, 8), torch.ones(2 * H * R * N, 8)
    yield "ssm_chunked_fwd", lambda **k: ops.chunked_fwd(x, B, B, s, s, s, th, **k), 2, 1
    yield "ssm_chunked_bwd", lambda **k: ops.chunked_bwd(x, B, B, s, s, s, th, x, **k), 8, 1
    yield "ssm_decode_step", lambda **k: ops.decode_step(h, *token, **k), 1, 0
    yield "rope_bc", lambda **k: ops.rope_bc(B, B, s, th, **k), 3, 1
    yield "bc_prologue", lambda **k: ops.bc_prologue(u, W, s, th, H, R, N, **k), 3, 1


ALL = [c if len(c) == 4 else c + (0 if c[0] == "layer_norm_fwd" else 1,) for c in (*block_calls(), *core_calls())]


@pytest.mark.parametrize("name,call,outputs,workspace", ALL, ids=[c[0] for c in ALL])
def test_allocations_belong_to_the_given_stream(fake, name, call, outputs, workspace):
    # a workspace that the call drops at return must not go back to another
    # stream's pool while the kernels on the given stream still use it
    seen = []

    class Allocations(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if func.overloadpacket.__name__ in ("empty", "empty_like", "new_empty", "empty_strided", "new_empty_strided"):
                seen.append(fake.inside)
            return func(*args, **(kwargs or {}))

    side = Stream()
    with Allocations():
        out = call(stream=side)
    assert len(seen) == outputs + workspace and all(s is side for s in seen)
    assert [c[0] for c in fake.calls] == ["mamba3_" + name]
    handle = fake.calls[0][1][-1]  # ... and the kernels go there
    assert getattr(handle, "value", handle) == side.cuda_stream
    # the outputs are read on the caller's stream next
    out = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else [out]
    mine = [t for t in out if t is not None]
    assert len(mine) == outputs and len(fake.recorded) == outputs
    assert all(a is b for a, b in zip(mine, fake.recorded))
    assert fake.inside is None


@pytest.mark.parametrize("call", [c[1] for c in ALL], ids=[c[0] for c in ALL])
def test_a_stream_of_another_device_is_refused(fake, call):
    class Other(Stream):
        device = torch.device("meta")

    with pytest.raises(ValueError, match="stream"):
        call(stream=Other())
    assert not fake.calls


@pytest.mark.parametrize("which", range(len(BLOCK)), ids=BLOCK)
def test_without_a_stream_the_current_one_is_used(fake, which):
    name, call, _ = list(block_calls())[which]
    call()
    assert fake.calls[0][0] == "mamba3_" + name and fake.calls[0][1][-1] == 0 and not fake.recorded


@pytest.mark.parametrize("which", range(1, len(BLOCK)), ids=BLOCK[1:])
def test_workspaces_that_are_refused(fake, which):
    # entries on top of each other (4096 counted, one there), every second byte, another device
    call = list(block_calls())[which][1]
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(4096), torch.zeros(8192, dtype=torch.uint8)[::2],
                torch.empty(4096, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=bad)
    assert not fake.calls
    # of any type, its size in bytes
    call(workspace=torch.zeros(1024))
    args = [getattr(a, "value", a) for a in fake.calls[0][1]]
    assert args[-2] == 4096


@pytest.mark.parametrize("shape", [(4, 16), (2, 2, 16), (4, 1, 16), (2, 1, 2, 16)])
def test_layer_norm_dx_has_the_shape_of_x(fake, shape):
    x, m = torch.ones(shape), torch.ones(4)
    wide = torch.zeros(4, 24)
    for skip, stride in ((None, 16), (x, 16), (x.view(4, 16), 16), (wide[:, 3:19], 24)):
        dx = ops.layer_norm_bwd(x, m, m, x, dskip=skip)["dx"]
        assert dx.shape == x.shape and dx.dtype == x.dtype
        # its rows lie where the kernel, which knows one stride, puts them
        assert dx.view(4, 16).stride() == (stride, 1)
        assert (fake.calls[-1][1][0].skip_stride or 16) == stride
        assert fake.calls[-1][1][7] == dx.data_ptr()
