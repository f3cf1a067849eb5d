"""The attention layer's operators in a row, as they are used: against the fp64
oracles, captured into a graph, on a stream of their own.  Needs an MI355X."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import attention as oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from state_space_sequence_03_amd import ops as o
    o.lib()
    return o


def host(t):
    return t.detach().double().cpu().numpy()


def test_a_row_of_them(ops):
    # fp32: norms and rotation, attention, and both backwards, against the
    # formulas in fp64 from end to end
    r = np.random.default_rng(1)
    L, Hq, Hk, D, window, sinks = 160, 6, 2, 64, 50, 3
    put = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()
    qkv, do = put(r.standard_normal((1, L, Hq + 2 * Hk, D))), put(r.standard_normal((1, L, Hq, D)))
    gq, gk = put(1 + 0.1 * r.standard_normal(D)), put(1 + 0.1 * r.standard_normal(D))
    theta, see = put(10000.0 ** (-np.arange(D // 2) * 2.0 / D)), {"window": window, "sinks": sinks}
    q0, k0, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
    q, k = ops.qk_norm_rope_fwd(q0, k0, gq, gk, theta=theta)
    o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = dqkv[:, :, :Hq], dqkv[:, :, Hq:Hq + Hk], dqkv[:, :, Hq + Hk:]
    ops.window_attn_bwd(q, k, v, o, lse, do, dq=dq, dk=dk, dv=dv, **see)
    g = ops.qk_norm_rope_bwd(q0, k0, dq, dk, gq, gk, theta=theta, dq=dq, dk=dk)
    h, pos, th = host(qkv[0]), np.arange(L), host(theta)
    a = [(h[:, :Hq], host(gq), 1e-5, th, pos, False), (h[:, Hq:Hq + Hk], host(gk), 1e-5, th, pos, False)]
    Q, K = (oracle.norm_rope(*x) for x in a)
    V, scale = h[:, Hq + Hk:], D ** -0.5
    O, lse64 = oracle.attention(Q, K, V, window, sinks, scale)
    dQ, dK, dV = oracle.attention_bwd(Q, K, V, O, lse64, host(do[0]), window, sinks, scale)
    (dQ, dGq), (dK, dGk) = oracle.norm_rope_bwd(*a[0], dQ), oracle.norm_rope_bwd(*a[1], dK)
    # each of the four steps is off by a few hundred units of 2^-23 of its own
    # magnitudes (D + 16 terms twice over, exponents of up to 8 + 8): 1e-4 of the
    # largest entry holds them all
    for name, got, want in (("o", o[0], O), ("lse", lse[0], lse64), ("dq", dq[0], dQ), ("dk", dk[0], dK), ("dv", dv[0], dV),
                            ("dgain_q", g["dgain_q"], dGq), ("dgain_k", g["dgain_k"], dGk)):
        off = np.abs(host(got) - want).max() / np.abs(want).max()
        assert off < 1e-4, (name, off)


def calls(ops):
    """Each entry point on operands of its own, with what it takes from its workspace."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()
    q, k, v, do = rand(2, 1500, 8, 64), rand(2, 1500, 2, 64), rand(2, 1500, 2, 64), rand(2, 1500, 8, 64)
    theta, see = torch.rand(32, device="cuda", generator=g), {"window": 100, "sinks": 4}
    o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
    kc, vc, lens = rand(1, 20000, 2, 64), rand(1, 20000, 2, 64), torch.tensor([19000], device="cuda")
    new = rand(1, 1, 8, 64), rand(1, 1, 2, 64), rand(1, 1, 2, 64)
    yield "qk_norm_rope_fwd", lambda **w: ops.qk_norm_rope_fwd(q, k, theta=theta, **w)
    yield "qk_norm_rope_bwd", lambda **w: ops.qk_norm_rope_bwd(q, k, do, v, theta=theta, **w)
    yield "window_attn_fwd", lambda **w: ops.window_attn_fwd(q, k, v, want_lse=True, **see, **w)
    yield "window_attn_bwd", lambda **w: ops.window_attn_bwd(q, k, v, o, lse, do, **see, **w)
    yield "window_attn_decode", lambda **w: ops.window_attn_decode(*new, kc, vc, lens, **w)


def tensors(out):
    return list(out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,))


def test_workspaces_outlive_their_call(ops):
    # the given stream is held up while the current one takes and overwrites
    # all the memory it can get
    side = torch.cuda.Stream()
    for name, call in calls(ops):
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


def test_two_streams_at_once(ops):
    # the same calls on two streams side by side, each with its own operands
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [list(calls(ops)) for _ in streams]
    want = [[[t.clone() for t in tensors(c())] for _, c in s] for s in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [[], []]
        for i in range(len(sets[0])):
            for n, s in enumerate(streams):
                got[n].append(tensors(sets[n][i][1](stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for p, w in zip(a, b) for x, y in zip(p, w))


def test_two_captured_steps(ops):
    # a training step of the layer in two graphs (equal and packed lengths),
    # each with its memory; replays in turn, with eager work between, equal eager
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).bfloat16()
    Hq, Hk, D, theta = 8, 2, 64, torch.rand(32, device="cuda", generator=g)
    sides = []
    for lead, starts in (((2, 700), None), ((1400,), torch.tensor([0, 5, 705, 1400], device="cuda"))):
        qkv, do = rand(*lead, Hq + 2 * Hk, D), rand(*lead, Hq, D)

        def step(qkv=qkv, do=do, see={"window": 90, "sinks": 3, "starts": starts}):
            q0, k0, v = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hk, :], qkv[..., Hq + Hk:, :]
            q, k = ops.qk_norm_rope_fwd(q0, k0, theta=theta)
            o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
            d = ops.window_attn_bwd(q, k, v, o, lse, do, **see)
            t = ops.qk_norm_rope_bwd(q0, k0, d["dq"], d["dk"], theta=theta)
            return [o, lse, t["dq"], t["dk"], d["dv"], t["dgain_q"], t["dgain_k"]]

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        sides.append((qkv, do, step, graph, out))
    for n in range(4):
        for qkv, do, step, graph, out in sides:
            qkv.copy_(rand(*qkv.shape))
            do.copy_(rand(*do.shape))
        want = [[t.clone() for t in s[2]()] for s in sides]
        torch.cuda.synchronize()
        for s in sides[::-1 if n % 2 else 1]:
            s[3].replay()
        torch.cuda.synchronize()
        for s, w in zip(sides, want):
            assert all(torch.equal(a, b) for a, b in zip(s[4], w)), n


def test_example(ops):
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    off, error = example.main()
    # bf16: outputs of size up to about 4 that differ by the rounding of q, k, o
    # and the product's sums, each 2^-8 of values of about 1
    assert off < 2e-2
    # fp32: third derivatives' part, about step^2 = 2^-16, and the sums' roundings over 2 step
    assert error < 5e-3


def test_rows_far_apart(ops):
    # the widest rows there may be, their bytes past 32 bits: as with contiguous rows, and nothing beside them written
    L, Hq, Hk, D, wide = 2200, 4, 2, 64, 1 << 20
    print(f"rows {wide} entries apart, {L} of them", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    rows = torch.zeros(L, wide, device="cuda", dtype=torch.bfloat16)
    at = iter(range(0, wide, 4096))

    def spot(heads, values=None):
        c = next(at)
        t = rows[:, c:c + heads * D].unflatten(1, (heads, D))[None]
        if values is not None:
            t.copy_(values)
        return t

    rand = lambda heads: torch.randn(1, L, heads, D, device="cuda", generator=g).bfloat16()
    q, k, v, do = rand(Hq), rand(Hk), rand(Hk), rand(Hq)
    turn = {"theta": torch.rand(D // 2, device="cuda", generator=g), "halves": True}
    see = {"window": 300, "sinks": 40}
    far = [spot(h, t) for h, t in ((Hq, q), (Hk, k), (Hk, v), (Hq, do))]
    spots = [spot(h) for h in (Hq, Hk, Hq, Hq, Hk, Hk, Hq, Hk)]
    qr, kr = ops.qk_norm_rope_fwd(q, k, **turn)
    ops.qk_norm_rope_fwd(far[0], far[1], q_out=spots[0], k_out=spots[1], **turn)
    o, lse = ops.window_attn_fwd(qr, kr, v, want_lse=True, **see)
    _, lse2 = ops.window_attn_fwd(spots[0], spots[1], far[2], o=spots[2], want_lse=True, **see)
    d = ops.window_attn_bwd(qr, kr, v, o, lse, do, **see)
    ops.window_attn_bwd(spots[0], spots[1], far[2], spots[2], lse2, far[3], dq=spots[3], dk=spots[4], dv=spots[5], **see)
    n = ops.qk_norm_rope_bwd(q, k, d["dq"], d["dk"], **turn)
    m = ops.qk_norm_rope_bwd(far[0], far[1], spots[3], spots[4], dq=spots[6], dk=spots[7], **turn)
    torch.cuda.synchronize()
    for got, want in zip(spots + [lse2, m["dgain_q"], m["dgain_k"]],
                         (qr, kr, o, d["dq"], d["dk"], d["dv"], n["dq"], n["dk"], lse, n["dgain_q"], n["dgain_k"])):
        assert torch.equal(got, want)
    for t in far + spots:
        t.zero_()
    assert not bool(rows.view(torch.int32).any())
    # a cache with slots as far apart
    caches = [spot(Hk, t) for t in (k, v)]
    plain = [k.clone(), v.clone()]
    new = [t[:, :5] for t in (q, k, v)]
    lens = torch.tensor([5 * L - 7], device="cuda")
    got = ops.window_attn_decode(*(t.contiguous() for t in new), *caches, lens, window=L - 100, sinks=40)
    want = ops.window_attn_decode(*(t.contiguous() for t in new), *plain, lens, window=L - 100, sinks=40)
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(caches, plain))
