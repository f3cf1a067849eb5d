"""The attention layer's calls in the binding, on the host: what they refuse, how
strides reach the library, where their allocations go.  No GPU and no launch:
the library is a stand-in that takes every call, and operands lie in host memory.
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


B, T, Hq, Hk, D, C = 2, 3, 4, 2, 16, 9
bf = torch.bfloat16


def heads(n, *lead, dtype=bf):
    return torch.zeros(*(lead or (B, T)), n, D, dtype=dtype)


def calls():
    """Each entry point: its name, the call, the outputs it makes itself, workspaces."""
    q, k, o, lse = heads(Hq), heads(Hk), heads(Hq), torch.zeros(B, T, Hq)
    g, th, cache, lens = torch.zeros(D), torch.zeros(D // 2), heads(Hk, B, C), torch.zeros(B, dtype=torch.int64)
    yield "qk_norm_rope_fwd", lambda **w: ops.qk_norm_rope_fwd(q, k, g, g, theta=th, **w), 2, 0
    yield "qk_norm_rope_bwd", lambda **w: ops.qk_norm_rope_bwd(q, k, q, k, g, g, theta=th, **w), 4, 1
    yield "window_attn_fwd", lambda **w: ops.window_attn_fwd(q, k, k, window=2, want_lse=True, **w), 2, 0
    yield "window_attn_bwd", lambda **w: ops.window_attn_bwd(q, k, k, o, lse, o, window=2, **w), 3, 1
    yield "window_attn_decode", lambda **w: ops.window_attn_decode(q, k, k, cache, cache, lens, **w), 1, 1


ALL = list(calls())
IDS = [c[0] for c in ALL]


@pytest.mark.parametrize("name,call,outputs,workspace", ALL, ids=IDS)
def test_allocations_belong_to_the_given_stream(fake, name, call, outputs, workspace):
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
    assert [c[0] for c in fake.calls] == ["mamba3_" + name] and fake.calls[0][1][-1] == side.cuda_stream
    out = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else [out]
    assert len(fake.recorded) == outputs and all(a is b for a, b in zip(out, fake.recorded))
    assert fake.inside is None
    with pytest.raises(ValueError, match="stream"):
        call(stream=type("Other", (Stream,), {"device": torch.device("meta")})())


@pytest.mark.parametrize("name,call,outputs,workspace", [c for c in ALL if c[3]], ids=[c[0] for c in ALL if c[3]])
def test_workspaces_that_are_refused(fake, name, call, outputs, workspace):
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(4096), torch.zeros(8192, dtype=torch.uint8)[::2],
                torch.empty(4096, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=bad)
    assert not fake.calls


def test_strides_reach_the_library(fake):
    qkv = torch.zeros(B, T, Hq + 2 * Hk, D, dtype=bf)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    wide = qkv.shape[2] * D
    ops.qk_norm_rope_fwd(q, k, q_out=q, k_out=k)
    d = fake.calls[-1][1][0]
    assert (d.rows, d.seqlen, d.q_heads, d.k_heads, d.head_dim, d.rope_dim) == (B * T, T, Hq, Hk, D, 0)
    assert (d.q_stride, d.k_stride, d.q_out_stride, d.k_out_stride) == (wide,) * 4
    ops.qk_norm_rope_bwd(q, k, heads(Hq), k, dk=k, want_dgain=False, theta=torch.zeros(3), halves=True)
    d = fake.calls[-1][1][0]
    assert (d.q_out_stride, d.k_out_stride, d.dq_stride, d.dk_stride, d.rope_dim, d.flags) == (0, wide, 0, wide, 6, ops.M3_FLAG_ROPE_HALVES)
    ops.window_attn_fwd(q, k, v, window=5, sinks=2, scale=0.5)
    d = fake.calls[-1][1][0]
    assert (d.batch, d.q_len, d.kv_len, d.kv_rows, d.window, d.sinks, d.scale, d.flags) == (B, T, T, 0, 5, 2, 0.5, 0)
    assert (d.q_stride, d.k_stride, d.v_stride, d.o_stride) == (wide, wide, wide, 0)
    ops.window_attn_fwd(q[0], k[0], v[0], starts=torch.tensor([0, 1, 3]))
    d = fake.calls[-1][1][0]
    assert (d.batch, d.rows, d.flags, d.q_stride) == (2, T, ops.M3_FLAG_PACKED, wide)
    # the first tokens of a cache of keys and values side by side
    cache = torch.zeros(B, C, 2 * Hk, D, dtype=bf)
    ops.window_attn_fwd(heads(Hq), cache[:, :5, :Hk], cache[:, :5, Hk:])
    d = fake.calls[-1][1][0]
    assert (d.kv_len, d.kv_rows, d.k_stride, d.v_stride) == (5, C, 2 * Hk * D, 2 * Hk * D)
    plain = heads(Hk, B, C)
    ops.window_attn_fwd(heads(Hq), plain[:, :5], plain[:, :5])
    d = fake.calls[-1][1][0]
    assert (d.kv_len, d.kv_rows, d.k_stride, d.v_stride) == (5, C, 0, 0)
    ops.window_attn_fwd(heads(Hq), plain[:, :1], plain[:, :1])
    d = fake.calls[-1][1][0]
    assert (d.kv_len, d.kv_rows) == (1, C)
    ops.window_attn_decode(q, k, v, cache[:, :, :Hk], cache[:, :, Hk:], torch.zeros(B, dtype=torch.int64), window=4, sinks=1)
    d = fake.calls[-1][1][0]
    assert (d.batch, d.tokens, d.capacity, d.k_cache_stride, d.q_stride) == (B, T, C, 2 * Hk * D, wide)
    # one token of each sequence: the distance between sequences is the tokens'
    one = torch.zeros(B, 1, Hq + 2 * Hk, D, dtype=bf)
    ops.window_attn_decode(one[:, :, :Hq], one[:, :, Hq:Hq + Hk], one[:, :, Hq + Hk:], plain, plain, torch.zeros(B, dtype=torch.int64))
    assert fake.calls[-1][1][0].q_stride == wide


def refused(kind, f, *a, **k):
    with pytest.raises(kind):
        f(*a, **k)


def test_norm_rope_refusals(fake):
    q, k, f = heads(Hq), heads(Hk), torch.float32
    for go in (ops.qk_norm_rope_fwd, lambda q, k, *a, **w: ops.qk_norm_rope_bwd(q, k, q, k, *a, **w)):
        refused(TypeError, go, q.half(), k.half())
        refused(TypeError, go, q, k.float())
        refused(ValueError, go, None, None)
        refused(ValueError, go, q, heads(Hk, B, T + 1))
        refused(ValueError, go, q, torch.zeros(B, T, Hk, 8, dtype=bf))
        refused(ValueError, go, q, k, torch.zeros(D - 1))
        refused(TypeError, go, q, k, torch.zeros(D, dtype=bf))
        refused(ValueError, go, q, k, None, torch.zeros(2, D))
        refused(ValueError, go, q, k, theta=torch.zeros(D // 2 + 1))
        refused(ValueError, go, q, k, theta=torch.zeros(2, 2))
        refused(TypeError, go, q, k, theta=torch.zeros(2, dtype=torch.float64))
        refused(TypeError, go, q, k, pos=torch.zeros(B, T, dtype=torch.int32))
        refused(ValueError, go, q, k, pos=torch.zeros(T, dtype=torch.int64))
        refused(ValueError, go, q.transpose(1, 2), k)                      # heads not side by side
        refused(ValueError, go, q[:, :, ::2], k)
        refused(ValueError, go, q[:, :1].expand(B, T, Hq, D), k)           # tokens on top of each other
        refused(ValueError, go, torch.zeros(2 * B, T, Hq, D, dtype=bf)[::2], k)  # tokens unevenly apart
        refused(ValueError, go, torch.zeros(Hq, D, dtype=bf), None)
    refused(ValueError, ops.qk_norm_rope_fwd, q, k, q_out=heads(Hk))
    refused(TypeError, ops.qk_norm_rope_fwd, q, k, k_out=k.float())
    refused(ValueError, ops.qk_norm_rope_bwd, q, k, None, k)
    refused(ValueError, ops.qk_norm_rope_bwd, q, k, q, q)
    refused(ValueError, ops.qk_norm_rope_bwd, q, k, q, k, dgain_q=torch.zeros(D + 1))
    refused(TypeError, ops.qk_norm_rope_bwd, q, k, q, k, dgain_k=torch.zeros(D, dtype=bf))
    assert not fake.calls


def test_attention_refusals(fake):
    q, k, o, lse = heads(Hq), heads(Hk), heads(Hq), torch.zeros(B, T, Hq)
    starts = torch.tensor([0, 1, 2])
    for go in (ops.window_attn_fwd, lambda q, k, v, **w: ops.window_attn_bwd(q, k, v, q, torch.zeros(q.shape[:-1]), q, **w)):
        refused(TypeError, go, q.half(), k.half(), k.half())
        refused(TypeError, go, q, k.float(), k)
        refused(ValueError, go, q, k, heads(Hq))
        refused(ValueError, go, q, heads(Hk, B + 1, T), heads(Hk, B + 1, T))
        refused(ValueError, go, q, torch.zeros(B, T, Hk, 8, dtype=bf), k)
        refused(ValueError, go, q[0], k[0], k[0])                          # packed without starts
        refused(ValueError, go, q, k, k, starts=starts)                    # starts with batches
        refused(ValueError, go, q[0], heads(Hk, T + 1), heads(Hk, T + 1), starts=starts)
        refused(TypeError, go, q[0], k[0], k[0], starts=starts.int())
        refused(ValueError, go, q[0], k[0], k[0], starts=starts[:0])
        refused(ValueError, go, q[0], k[0], k[0], starts=torch.zeros(2, 2, dtype=torch.int64))
        refused(ValueError, go, q.transpose(1, 2), k, k)
        refused(ValueError, go, q, heads(Hk, B, C)[:, :T], k)              # k part of a cache, v not
    refused(ValueError, ops.window_attn_fwd, q, k, k, o=heads(Hk))
    refused(ValueError, ops.window_attn_fwd, q, k, k, lse=torch.zeros(B, Hq, T))
    refused(TypeError, ops.window_attn_fwd, q, k, k, lse=lse.to(bf))
    refused(ValueError, ops.window_attn_bwd, q, k, k, o, None, o)
    refused(ValueError, ops.window_attn_bwd, q, k, k, heads(Hk), lse, o)
    refused(ValueError, ops.window_attn_bwd, q, k, k, o, lse, o, dk=o)
    part = heads(Hk, B, C)[:, :T]
    refused(ValueError, ops.window_attn_bwd, q, part, part, o, lse, o)     # gradients of a cache's tokens
    assert not fake.calls
    out = ops.window_attn_bwd(q, part, part, o, lse, o, want_dk=False, want_dv=False)
    assert set(out) == {"dq"} and len(fake.calls) == 1


def test_decode_refusals(fake):
    q, k, cache, lens = heads(Hq), heads(Hk), heads(Hk, B, C), torch.zeros(B, dtype=torch.int64)
    go = ops.window_attn_decode
    refused(TypeError, go, q.half(), k.half(), k.half(), cache.half(), cache.half(), lens)
    refused(TypeError, go, q, k, k, cache.float(), cache, lens)
    refused(TypeError, go, q, k, k, cache, cache, lens.int())
    refused(ValueError, go, q, k, k, cache, cache, lens[:1])
    refused(ValueError, go, q, k[:, :2], k, cache, cache, lens)
    refused(ValueError, go, q, k, k[:, :2], cache, cache, lens)
    refused(ValueError, go, q, k, k, cache[:1], cache[:1], lens)
    refused(ValueError, go, q, k, k, cache, heads(Hk, B, C + 1), lens)
    refused(ValueError, go, q, k, k, heads(Hq, B, C), heads(Hq, B, C), lens)
    refused(ValueError, go, q, k, k, heads(Hk, B, 2 * C)[:, ::2][:, :C][:, :, :1], cache, lens)
    refused(ValueError, go, q, k, k, heads(Hk, B, 2 * C)[:, :C], heads(Hk, B, 2 * C)[:, :C], lens)  # part of a longer one
    refused(ValueError, go, q[0], k[0], k[0], cache, cache, lens)
    refused(ValueError, go, q, k, k, cache, cache, lens, o=heads(Hk))
    assert not fake.calls


def test_slots(fake):
    got = ops.window_cache_slots(torch.arange(12), 2, 7)
    assert got.tolist() == [0, 1, 2, 3, 4, 5, 6, 2, 3, 4, 5, 6]


def test_single_tokens_of_a_projection(fake):
    # sequences of one token each: slices of a projection's heads are evenly spaced tokens, not parts of a cache
    qkv = heads(Hq + 2 * Hk, B, 1)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    width = (Hq + 2 * Hk) * D
    single = qkv[:, 0, Hq:Hq + Hk].unsqueeze(1)
    for keys, stride in ((k, width), (heads(Hk, B, 1), 0), (single, width)):
        o, lse = ops.window_attn_fwd(q, keys, v, want_lse=True)
        assert set(ops.window_attn_bwd(q, keys, v, o, lse, o)) == {"dq", "dk", "dv"}
        for name, args in fake.calls:
            dims = args[0]
            assert (dims.q_stride, dims.k_stride, dims.v_stride, dims.kv_rows) == (width, stride, width, 0), name
        fake.calls.clear()
    # the first tokens of caches too long for that: rows from sequence to sequence
    cache = torch.empty_strided((B, 1, Hk, D), (1 << 21, Hk * D, D, 1), dtype=bf)
    ops.window_attn_fwd(q, cache, cache)
    dims = fake.calls[0][1][0]
    assert dims.kv_rows == (1 << 21) // (Hk * D) and dims.k_stride in (0, Hk * D)


# heads of a row, those taken, slots of a cache: the distance of the sequences is a multiple of the row taken or not
@pytest.mark.parametrize("all_heads,taken,slots", [(7, 2, 5), (6, 4, 3), (5, 3, 5), (3, 2, 3), (5, 2, 5), (8, 2, 9), (2, 2, 9)])
@pytest.mark.parametrize("length", [1, 2])
def test_sequences_lie_where_their_keys_do(fake, all_heads, taken, slots, length):
    # the first tokens of a cache of wider rows: what the library is told leads to every sequence's first key
    n = 3
    cache = heads(all_heads, n, slots)
    wide = heads(all_heads * slots, n, 1)  # the same memory layout, single tokens of very wide rows
    q = heads(2 * taken, n, length)
    for keys in ([cache[:, :length, :taken], cache[:, :length, -taken:]],
                 [wide[:, :, :taken], wide[:, :, -taken:]] if length == 1 else []):
        if not keys:
            continue
        k, v = keys
        o, lse = ops.window_attn_fwd(q, k, v, want_lse=True)
        ops.window_attn_bwd(q, k, v, o, lse, o, want_dk=False, want_dv=False)
        for name, args in fake.calls:
            dims = args[0]
            for stride in (dims.k_stride, dims.v_stride):
                assert (dims.kv_rows or length) * (stride or taken * D) == k.stride(0) == v.stride(0), name
        fake.calls.clear()


def test_single_keys_too_far_apart(fake):
    # a distance past the widest row there may be: by the rows it divides into, or else as evenly spaced tokens, whose
    # stride the library refuses
    row, q = Hk * D, heads(Hq, B, 1)
    for step, between in ((3 * row, 3 * row << 16), (3 * row + 8, (3 * row + 8) << 16), (1 << 21, 1 << 22), (3 * row, (1 << 21) + 8)):
        k = torch.empty_strided((B, 1, Hk, D), (between, step, D, 1), dtype=bf)
        ops.window_attn_fwd(q, k, k)
        dims = fake.calls[-1][1][0]
        assert (dims.kv_rows or 1) * (dims.k_stride or row) == between
        assert dims.k_stride <= 1 << 20 or dims.kv_rows == 0


def test_slots_of_a_cache_without_a_ring(fake):
    # refused on the host: the remainder by 0 or less would give slots outside the cache
    for sinks, capacity in ((4, 4), (5, 4), (0, 0), (-1, 4)):
        refused(ValueError, ops.window_cache_slots, torch.arange(3), sinks, capacity)
    assert ops.window_cache_slots(torch.arange(5), 3, 4).tolist() == [0, 1, 2, 3, 3]
