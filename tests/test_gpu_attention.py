"""Parity of windowed attention with sinks, forward and backward, with its fp64
oracle (oracle/attention.py, pinned in tests/test_oracle_attention_pins.py).
Needs an MI355X.  Every output entry is held to the oracle's bound for it."""
import numpy as np
import pytest

from oracle import attention as oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# half a step of the outputs' type, and of p and ds as the products take them
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from state_space_sequence_03_amd import ops as o
    o.lib()
    return o


def host(t):
    return t.detach().double().cpu().numpy()


def draw(rng, shape, io, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda().to(IO[io])


def within(name, got, ref, bound):
    got = host(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - ref) <= bound) | (got == ref))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} entries off, first {i}: {got[i]} against {ref[i]}, "
                             f"bound {np.broadcast_to(bound, ref.shape)[i]}")


def check_forward(io, o, lse, q, k, v, window, sinks, scale, what=""):
    """One sequence's outputs against the oracle."""
    u = HALF_STEP[io]
    a = (host(q), host(k), host(v), window, sinks, scale)
    for name, got, want, bound in zip(("o", "lse"), (o, lse), oracle.attention(*a), oracle.attention_bound(*a, u, u)):
        within(f"{what} {name}", got, want, bound)


def check_backward(io, grads, q, k, v, o, lse, do, window, sinks, scale, what=""):
    u = HALF_STEP[io]
    a = tuple(host(t) for t in (q, k, v, o, lse, do)) + (window, sinks, scale)
    for name, got, want, bound in zip(("dq", "dk", "dv"), grads, oracle.attention_bwd(*a),
                                      oracle.attention_bwd_bound(*a, u, u)):
        within(f"{what} {name}", got, want, bound)


# q_len, kv_len, q_heads, kv_heads, D, window, sinks
SHAPES = [
    (1, 1, 1, 1, 8, 0, 0), (5, 5, 2, 1, 24, 0, 0), (33, 33, 3, 3, 32, 7, 2), (64, 64, 4, 2, 64, 64, 1),
    (65, 65, 2, 2, 72, 1, 0), (128, 128, 2, 1, 128, 0, 0), (129, 129, 6, 2, 96, 32, 5), (300, 300, 4, 1, 128, 40, 3),
    (300, 300, 5, 5, 40, 64, 70), (257, 257, 2, 2, 64, 100, 300), (200, 450, 4, 2, 64, 60, 4), (1, 300, 8, 2, 128, 33, 1),
    (17, 1000, 2, 1, 80, 0, 0), (450, 200, 2, 1, 64, 50, 3), (300, 40, 2, 2, 128, 0, 0), (700, 700, 2, 1, 64, 130, 130),
    (1100, 1100, 2, 2, 64, 20, 4), (1500, 1500, 2, 1, 128, 100, 200), (1300, 1700, 1, 1, 32, 30, 1),
]


@pytest.mark.parametrize("n,m,Hq,Hk,D,window,sinks", SHAPES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_against_the_oracle(ops, io, n, m, Hq, Hk, D, window, sinks):
    print(f"attention {io} {n} of {m}, heads {Hq}/{Hk} x {D}, window {window} sinks {sinks}", flush=True)
    r = np.random.default_rng(n + m + D)
    q, k, v, do = (draw(r, (2, l, h, D), io) for l, h in ((n, Hq), (m, Hk), (m, Hk), (n, Hq)))
    scale = D ** -0.5
    see = {"window": window, "sinks": sinks}
    o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
    torch.cuda.synchronize()
    for b in range(2):
        check_forward(io, o[b], lse[b], q[b], k[b], v[b], window, sinks, float(np.float32(scale)), b)
    g = ops.window_attn_bwd(q, k, v, o, lse, do, **see)
    torch.cuda.synchronize()
    assert set(g) == {"dq", "dk", "dv"}
    for b in range(2):
        check_backward(io, [g[x][b] for x in ("dq", "dk", "dv")], q[b], k[b], v[b], o[b], lse[b], do[b], window, sinks,
                       float(np.float32(scale)), b)
    # any subset of the gradients, and a forward without statistics: the same values
    one = ops.window_attn_bwd(q, k, v, o, lse, do, want_dq=False, want_dk=False, **see)
    assert set(one) == {"dv"} and torch.equal(one["dv"], g["dv"])
    one = ops.window_attn_bwd(q, k, v, o, lse, do, want_dk=False, want_dv=False, **see)
    assert set(one) == {"dq"} and torch.equal(one["dq"], g["dq"])
    assert torch.equal(ops.window_attn_fwd(q, k, v, **see)[0], o)


PACKED = [([1], 0, 0, 64), ([5, 1, 200, 64, 1], 50, 3, 64), ([130, 0, 0, 129, 128, 3], 0, 0, 128),
          ([1] * 70 + [300] + [2] * 70, 40, 5, 32), ([1200, 7, 1030, 1024], 60, 2, 64), ([0, 0, 40], 9, 150, 72)]


@pytest.mark.parametrize("lens,window,sinks,D", PACKED)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_packed_sequences(ops, io, lens, window, sinks, D):
    # every sequence by itself, and the rows before the first and behind the last left as they were
    print(f"packed {io} {len(lens)} sequences", flush=True)
    Hq, Hk, before, behind = 4, 2, 3, 70
    rows = before + sum(lens) + behind
    r = np.random.default_rng(rows)
    q, k, v, do = (draw(r, (rows, h, D), io) for h in (Hq, Hk, Hk, Hq))
    ends = [before]
    for n in lens:
        ends.append(ends[-1] + n)
    for t in (q, k, v, do):
        t[:before] = t[ends[-1]:] = float("nan")
    starts = torch.tensor(ends, device="cuda")
    see = {"window": window, "sinks": sinks, "starts": starts, "scale": 0.25}
    o, lse = torch.full_like(q, 5.0), torch.full((rows, Hq), 5.0, device="cuda")
    ops.window_attn_fwd(q, k, v, o=o, lse=lse, **see)
    out = {"dq": torch.full_like(q, 5.0), "dk": torch.full_like(k, 5.0), "dv": torch.full_like(v, 5.0)}
    g = ops.window_attn_bwd(q, k, v, o, lse, do, **see, **out)
    torch.cuda.synchronize()
    for a, b in zip(ends, ends[1:]):
        if a < b:
            s = slice(a, b)
            check_forward(io, o[s], lse[s], q[s], k[s], v[s], window, sinks, 0.25, (a, b))
            check_backward(io, [g[x][s] for x in ("dq", "dk", "dv")], q[s], k[s], v[s], o[s], lse[s], do[s], window, sinks,
                           0.25, (a, b))
    for t in (o, lse, g["dq"], g["dk"], g["dv"]):
        assert bool((t[:before] == 5.0).all()) and bool((t[ends[-1]:] == 5.0).all())


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_slices_of_a_projection(ops, io):
    # q, k, v and their gradients as slices of rows of all heads, o beside something else
    r = np.random.default_rng(11)
    B, L, Hq, Hk, D = 2, 150, 4, 2, 64
    qkv = draw(r, (B, L, Hq + 2 * Hk, D), io)
    cut = lambda t: (t[:, :, :Hq], t[:, :, Hq:Hq + Hk], t[:, :, Hq + Hk:])
    see = {"window": 60, "sinks": 2}
    q, k, v = cut(qkv)
    o, lse = ops.window_attn_fwd(*(t.contiguous() for t in (q, k, v)), want_lse=True, **see)
    wide = torch.full((B, L, Hq + 1, D), float("nan"), dtype=IO[io], device="cuda")
    ops.window_attn_fwd(q, k, v, o=wide[:, :, 1:], **see)
    assert torch.equal(wide[:, :, 1:], o) and bool(wide[:, :, 0].isnan().all())
    do = draw(r, (B, L, Hq, D), io)
    g = ops.window_attn_bwd(*(t.contiguous() for t in (q, k, v)), o, lse, do, **see)
    wide_do = torch.zeros((B, L, Hq + 1, D), dtype=IO[io], device="cuda")
    wide_do[:, :, :Hq] = do
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = cut(dqkv)
    ops.window_attn_bwd(q, k, v, wide[:, :, 1:], lse, wide_do[:, :, :Hq], dq=dq, dk=dk, dv=dv, **see)
    assert torch.equal(dqkv, torch.cat((g["dq"], g["dk"], g["dv"]), 2))


def test_keys_of_a_longer_cache(ops):
    # the first tokens of a cache as keys: what lies behind them is not read
    r = np.random.default_rng(12)
    cache = [draw(r, (3, 400, 2, 64), "bf16") for _ in range(2)]
    for t in cache:
        t[:, 210:] = float("nan")
    q = draw(r, (3, 50, 4, 64), "bf16")
    k, v = (t[:, :210] for t in cache)
    want, _ = ops.window_attn_fwd(q, k.contiguous(), v.contiguous(), window=70, sinks=3)
    got, _ = ops.window_attn_fwd(q, k, v, window=70, sinks=3)
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("n,m,window,sinks", [(300, 300, 40, 3), (40, 90, 0, 0), (700, 700, 60, 3)])
def test_gradients_laid_out_as_a_cache(ops, n, m, window, sinks):
    # the library's own call with kv_rows above kv_len: dk and dv lie as k and v do, their other rows stay as they were
    r = np.random.default_rng(16)
    B, Hq, Hk, D, rows = 2, 4, 2, 64, m + 37
    q, do = draw(r, (B, n, Hq, D), "bf16"), draw(r, (B, n, Hq, D), "bf16")
    k, v = draw(r, (B, rows, Hk, D), "bf16"), draw(r, (B, rows, Hk, D), "bf16")
    k[:, m:] = v[:, m:] = float("nan")
    see = {"window": window, "sinks": sinks, "scale": 0.125}
    o, lse = ops.window_attn_fwd(q, k[:, :m], v[:, :m], want_lse=True, **see)
    want = ops.window_attn_bwd(q, k[:, :m].contiguous(), v[:, :m].contiguous(), o, lse, do, **see)
    dims = ops.AttnDims(batch=B, q_len=n, kv_len=m, kv_rows=rows, q_heads=Hq, kv_heads=Hk, head_dim=D, io_dtype=ops.M3_BF16,
                        **see)
    out = [torch.full_like(t, 5.0) for t in (q, k, v)]
    memory = torch.empty(ops.window_attn_bwd_workspace_size(dims), dtype=torch.uint8, device="cuda")
    at = [t.data_ptr() for t in (q, k, v, o, lse, do)]
    st = ops.lib().mamba3_window_attn_bwd(dims, *at, None, *(t.data_ptr() for t in out), memory.data_ptr(), memory.numel(),
                                          torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == ops.M3_OK and torch.equal(out[0], want["dq"])
    assert torch.equal(out[1][:, :m], want["dk"]) and torch.equal(out[2][:, :m], want["dv"])
    assert bool((out[1][:, m:] == 5.0).all()) and bool((out[2][:, m:] == 5.0).all())


@pytest.mark.parametrize("all_heads,taken,slots", [(7, 2, 5), (6, 4, 3), (5, 3, 5), (3, 2, 3), (8, 2, 9)])
def test_first_keys_of_a_cache(ops, all_heads, taken, slots):
    # one key of each sequence, the sequences a whole number of its row apart or not: as with contiguous keys
    r = np.random.default_rng(17)
    kv = draw(r, (4, slots, all_heads, 64), "bf16")
    q, do = draw(r, (4, 3, 2 * taken, 64), "bf16"), draw(r, (4, 3, 2 * taken, 64), "bf16")
    k, v = kv[:, :1, :taken], kv[:, :1, -taken:]
    plain = k.contiguous(), v.contiguous()
    want, lse = ops.window_attn_fwd(q, *plain, want_lse=True)
    got, lse2 = ops.window_attn_fwd(q, k, v, want_lse=True)
    assert torch.equal(got, want) and torch.equal(lse2, lse) and torch.equal(got[:, 2, ::2], v[:, 0])
    g, h = ops.window_attn_bwd(q, *plain, want, lse, do), ops.window_attn_bwd(q, k, v, got, lse2, do)
    assert all(torch.equal(g[n], h[n]) for n in g)
    one = ops.window_attn_bwd(q, k, v, got, lse2, do, want_dk=False, want_dv=False)
    assert torch.equal(one["dq"], g["dq"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_large_scores(ops, io):
    # softmaxes that are nearly one-hot, rising and falling along the keys; the
    # running maximum moves by far more than what it is let behind by
    r = np.random.default_rng(13)
    L, D = 400, 64
    q, v, do = (draw(r, (1, L, 2, D), io) for _ in range(3))
    for ramp in (np.linspace(0.2, 12, L), np.linspace(12, 0.2, L)):
        k = (draw(r, (1, L, 2, D), "f32") * torch.from_numpy(ramp.astype(np.float32)).cuda()[None, :, None, None]).to(IO[io])
        o, lse = ops.window_attn_fwd(q, k, v, window=333, sinks=1, want_lse=True, scale=1.0)
        check_forward(io, o[0], lse[0], q[0], k[0], v[0], 333, 1, 1.0)
        g = ops.window_attn_bwd(q, k, v, o, lse, do, window=333, sinks=1, scale=1.0)
        check_backward(io, [g[x][0] for x in ("dq", "dk", "dv")], q[0], k[0], v[0], o[0], lse[0], do[0], 333, 1, 1.0)


def test_gradients_against_differences(ops):
    # fp32: directional differences of the forward itself, in fp64 sums
    r = np.random.default_rng(14)
    L, D = 200, 32
    q, k, v, do = (draw(r, (1, L, h, D), "f32") for h in (4, 2, 2, 4))
    see = {"window": 50, "sinks": 2}
    loss = lambda *a: float((ops.window_attn_fwd(*a, **see)[0].double() * do.double()).sum())
    o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
    g = ops.window_attn_bwd(q, k, v, o, lse, do, **see)
    for i, n in enumerate(("dq", "dk", "dv")):
        d = draw(r, tuple((q, k, v)[i].shape), "f32")
        step = 2.0 ** -7
        shifted = [[t + s * step * d if j == i else t for j, t in enumerate((q, k, v))] for s in (1, -1)]
        quotient = (loss(*shifted[0]) - loss(*shifted[1])) / (2 * step)
        slope = float((g[n].double() * d.double()).sum())
        # the sums of both losses carry 25600 terms' fp32 errors of about 2e-7
        # each: 25600^(1/2) 3e-7 / step = 6e-3; the third derivatives' part,
        # step^2 / 6 of a slope's size, is 1e-5 of it
        assert abs(quotient - slope) < 2e-2 + 1e-3 * abs(slope), (n, quotient, slope)


def test_small_calls(ops):
    empty = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    o, lse = ops.window_attn_fwd(empty(0, 7, 2, 64), empty(0, 7, 1, 64), empty(0, 7, 1, 64), want_lse=True)
    assert o.shape == (0, 7, 2, 64) and lse.shape == (0, 7, 2)
    # no queries: keys still get their zero gradients; no keys: outputs are zero
    k = torch.ones((2, 9, 1, 64), dtype=torch.bfloat16, device="cuda")
    q0 = empty(2, 0, 2, 64)
    o, lse = ops.window_attn_fwd(q0, k, k, want_lse=True)
    g = ops.window_attn_bwd(q0, k, k, o, lse, q0)
    assert g["dq"].shape == q0.shape and not bool(g["dk"].any()) and not bool(g["dv"].any())
    q = torch.ones((2, 9, 2, 64), dtype=torch.bfloat16, device="cuda")
    k0 = empty(2, 0, 1, 64)
    o, lse = ops.window_attn_fwd(q, k0, k0, want_lse=True)
    assert not bool(o.any()) and bool((lse == -float("inf")).all())
    assert not bool(ops.window_attn_bwd(q, k0, k0, o, lse, q)["dq"].any())


def test_repeats_bit_for_bit(ops):
    r = np.random.default_rng(15)
    q, k, v, do = (draw(r, (2, 1400, h, 64), "bf16") for h in (8, 2, 2, 8))
    see = {"window": 90, "sinks": 4}
    o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
    g = ops.window_attn_bwd(q, k, v, o, lse, do, **see)
    for _ in range(3):
        p, l = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
        assert torch.equal(p, o) and torch.equal(l, lse)
        h = ops.window_attn_bwd(q, k, v, o, lse, do, **see)
        assert all(torch.equal(h[n], g[n]) for n in g)


# batch, q_len, kv_len, q_heads, kv_heads, D, window, sinks: few blocks of queries
# (with more than 512 keys each: in parts), and enough to occupy the chip
SIZES = [
    (1, 700, 700, 4, 1, 64, 600, 40), (1, 640, 1300, 4, 2, 128, 513, 33), (2, 577, 577, 3, 3, 96, 0, 0),
    (1, 130, 901, 2, 2, 32, 800, 100), (1, 40, 1999, 8, 2, 128, 1500, 65), (1, 700, 600, 6, 2, 72, 0, 0),
    (14, 300, 300, 8, 2, 64, 70, 33), (9, 650, 700, 5, 5, 40, 96, 1), (13, 260, 500, 14, 7, 128, 130, 64),
    (70, 65, 65, 4, 2, 96, 0, 0),
]


@pytest.mark.parametrize("B,n,m,Hq,Hk,D,window,sinks", SIZES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_few_blocks_and_many(ops, io, B, n, m, Hq, Hk, D, window, sinks):
    print(f"attention {io} {B} x {n} of {m}, heads {Hq}/{Hk} x {D}, window {window} sinks {sinks}", flush=True)
    r = np.random.default_rng(n + m + D)
    q, k, v, do = (draw(r, (B, l, h, D), io) for l, h in ((n, Hq), (m, Hk), (m, Hk), (n, Hq)))
    see = {"window": window, "sinks": sinks, "scale": 0.125}
    o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
    g = ops.window_attn_bwd(q, k, v, o, lse, do, **see)
    torch.cuda.synchronize()
    for b in {0, B // 2, B - 1}:
        a = window, sinks, 0.125, b
        check_forward(io, o[b], lse[b], q[b], k[b], v[b], *a)
        check_backward(io, [g[x][b] for x in ("dq", "dk", "dv")], q[b], k[b], v[b], o[b], lse[b], do[b], *a)
    assert torch.equal(ops.window_attn_fwd(q, k, v, **see)[0], o)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_large_scores_in_parts(ops, io, D):
    # one part's scores far above the other's: the sharp end comes first, last, and in turns of 64 keys
    r = np.random.default_rng(D)
    L = 900
    turns = np.where(np.arange(L) // 64 % 2 == 0, 0.1, 10.0)
    q, v, do = (draw(r, (1, L, 2, D), io) for _ in range(3))
    for ramp in (np.linspace(0.2, 12, L), np.linspace(12, 0.2, L), turns, 10.1 - turns):
        k = (draw(r, (1, L, 2, D), "f32") * torch.from_numpy(ramp.astype(np.float32)).cuda()[None, :, None, None]).to(IO[io])
        for window, sinks in ((0, 0), (600, 33)):
            see = {"window": window, "sinks": sinks, "scale": 1.0}
            o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
            check_forward(io, o[0], lse[0], q[0], k[0], v[0], window, sinks, 1.0)
            g = ops.window_attn_bwd(q, k, v, o, lse, do, **see)
            check_backward(io, [g[x][0] for x in ("dq", "dk", "dv")], q[0], k[0], v[0], o[0], lse[0], do[0], window, sinks, 1.0)


@pytest.mark.parametrize("lens,window,sinks,D", [([700, 1, 600, 0, 64], 0, 0, 64), ([900, 40, 530], 600, 33, 128),
                                                 ([1], 0, 0, 32), ([513, 5], 1024, 3, 96)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_packed_sequences_in_parts(ops, io, lens, window, sinks, D):
    test_packed_sequences(ops, io, lens, window, sinks, D)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_starts_that_do_not_rise(ops, io):
    # 24 pieces of 256 queries where 3 sequences of 3000 rows have 14 at most: the call stays within its workspace, and what it does
    # not write there it does not read
    rows, heads, D = 3000, 8, 64
    print(f"starts that fall {io} {rows} rows", flush=True)
    r = np.random.default_rng(18)
    q, k, v, do = (draw(r, (rows, heads, D), io) for _ in range(4))
    starts = torch.tensor([0, rows, 0, rows], device="cuda")
    dims = ops.AttnDims(batch=3, rows=rows, q_heads=heads, kv_heads=heads, head_dim=D, window=20, sinks=4, scale=0.125,
                        io_dtype=ops.M3_BF16 if io == "bf16" else ops.M3_F32, flags=ops.M3_FLAG_PACKED)
    need = ops.window_attn_bwd_workspace_size(dims)
    memory = torch.full((2 * need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN, read as fp32
    see = {"window": 20, "sinks": 4, "scale": 0.125, "starts": starts}
    o, lse = ops.window_attn_fwd(q, k, v, want_lse=True, **see)
    g = ops.window_attn_bwd(q, k, v, o, lse, do, workspace=memory[:need], **see)
    torch.cuda.synchronize()
    assert bool((memory[need:] == 0xFF).all())
    assert all(bool(torch.isfinite(t).all()) for t in (o, lse, *g.values()))
