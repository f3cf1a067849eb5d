"""Attention of new tokens over a cache that wraps, against the fp64 oracle
(oracle/attention.py) of the whole sequences.  Needs an MI355X."""
import numpy as np
import pytest

from oracle import attention as oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

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


def draw(rng, shape, io):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(IO[io])


def within(name, got, ref, bound):
    got = host(got)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} entries off, first {i}: {got[i]} against {ref[i]}, "
                             f"bound {np.broadcast_to(bound, ref.shape)[i]}")


def cached(ops, k, length, sinks, capacity):
    """A cache that `length` tokens of k were written to one by one; NaN where none lies."""
    cache = torch.full((capacity,) + tuple(k.shape[1:]), float("nan"), dtype=k.dtype, device="cuda")
    for p in range(length):
        cache[oracle.slot(p, sinks, capacity)] = k[p]
    return cache


# tokens, q_heads, kv_heads, D, window, sinks, capacity, lengths before the call
CASES = [
    (1, 1, 1, 8, 0, 0, 5, [0, 4]),
    (1, 4, 1, 64, 0, 0, 40, [0, 1, 31, 39]),
    (1, 16, 4, 128, 32, 4, 36, [0, 3, 35, 36, 37, 500]),
    (1, 4, 4, 72, 100, 0, 100, [99, 100, 163, 250]),
    (1, 40, 1, 64, 60, 2, 70, [10, 69, 70, 200]),
    (3, 4, 2, 64, 33, 5, 40, [0, 2, 4, 35, 40, 41, 300]),
    (16, 8, 2, 128, 64, 4, 83, [0, 70, 83, 90, 1000]),
    (16, 5, 5, 32, 20, 130, 165, [0, 100, 129, 130, 140, 900]),
    (5, 8, 8, 40, 1, 0, 5, [0, 3, 5, 77]),
    (2, 2, 1, 64, 0, 3, 50, [47, 48, 49, 120]),        # no window, wrapped: what the cache holds
    (1, 2, 1, 96, 10, 1, 300, [0, 9, 10, 150, 299, 300, 700]),  # a cache far longer than the window
    (1, 8, 1, 128, 0, 0, 3000, [0, 2000, 2999]),       # split over blocks
    (4, 8, 2, 64, 2500, 7, 2600, [1, 1500, 2590, 2600, 9000]),
]


@pytest.mark.parametrize("T,Hq,Hk,D,window,sinks,capacity,lens", CASES)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_against_the_oracle(ops, io, T, Hq, Hk, D, window, sinks, capacity, lens):
    print(f"decode {io} T {T} heads {Hq}/{Hk} x {D} window {window} sinks {sinks} capacity {capacity}", flush=True)
    r = np.random.default_rng(capacity + T)
    B, longest = len(lens), max(lens) + T
    k, v = draw(r, (B, longest, Hk, D), io), draw(r, (B, longest, Hk, D), io)
    q = draw(r, (B, T, Hq, D), io)
    kc, vc = (torch.stack([cached(ops, t[b], n, sinks, capacity) for b, n in enumerate(lens)]) for t in (k, v))
    new = [torch.stack([t[b, n:n + T] for b, n in enumerate(lens)]) for t in (k, v)]
    want_cache = [torch.stack([cached(ops, t[b], n + T, sinks, capacity) for b, n in enumerate(lens)]) for t in (k, v)]
    n = torch.tensor(lens, device="cuda")
    o = ops.window_attn_decode(q, *new, kc, vc, n, window=window, sinks=sinks, scale=0.2)
    torch.cuda.synchronize()
    for got, want in zip((kc, vc), want_cache):
        assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))
    u = HALF_STEP[io]
    for b, m in enumerate(lens):
        see = oracle.decode_visible(m + T, T, window, sinks, capacity)
        a = (host(q[b]), host(k[b, :m + T]), host(v[b, :m + T]), window, sinks, float(np.float32(0.2)))
        within(f"sequence of {m}", o[b], oracle.attention(*a, see)[0], oracle.attention_bound(*a, u, u, see)[0])
    # again on the cache it has written: the same
    assert torch.equal(ops.window_attn_decode(q, *new, kc, vc, n, window=window, sinks=sinks, scale=0.2), o)


def test_idle_sequences(ops):
    r = np.random.default_rng(2)
    q, k, v = draw(r, (3, 2, 4, 64), "bf16"), draw(r, (3, 2, 2, 64), "bf16"), draw(r, (3, 2, 2, 64), "bf16")
    for capacity in (40, 4000):  # one block, split over blocks
        kc, vc = draw(r, (3, capacity, 2, 64), "bf16"), draw(r, (3, capacity, 2, 64), "bf16")
        before = kc.clone(), vc.clone()
        o = ops.window_attn_decode(q, k, v, kc, vc, torch.tensor([5, -1, 9], device="cuda"))
        assert not bool(o[1].any()) and bool(o[0].any()) and bool(o[2].any())
        assert torch.equal(kc[1], before[0][1]) and torch.equal(vc[1], before[1][1])
        assert torch.equal(kc[0, 5:7], k[0]) and torch.equal(vc[2, 9:11], v[2])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_generation_follows_the_prefill(ops, io):
    # a prompt, its cache filled by slots, then tokens one by one and in groups:
    # the same as one forward over everything
    r = np.random.default_rng(3)
    B, L, Hq, Hk, D, window, sinks, capacity = 2, 150, 4, 2, 64, 48, 3, 60
    q, k, v = (draw(r, (B, L, h, D), io) for h in (Hq, Hk, Hk))
    whole, _ = ops.window_attn_fwd(q, k, v, window=window, sinks=sinks)
    prompt = 70
    kc, vc = (torch.full((B, capacity, Hk, D), float("nan"), dtype=IO[io], device="cuda") for _ in range(2))
    keep = torch.tensor(oracle.held(prompt, sinks, capacity), device="cuda")
    at = ops.window_cache_slots(keep, sinks, capacity)
    kc[:, at], vc[:, at] = k[:, keep], v[:, keep]
    lens = torch.full((B,), prompt, device="cuda")
    p = prompt
    for T in (1, 1, 5, 1, 10, 7, 9, 1, 1, 10, 10, 10, 9, 5):
        cut = [t[:, p:p + T] for t in (q, k, v)]
        o = ops.window_attn_decode(cut[0].contiguous(), cut[1].contiguous(), cut[2].contiguous(), kc, vc, lens, window=window,
                                   sinks=sinks)
        a = (whole[:, p:p + T].double() - o.double()).abs()
        # two results, each within its own bound of the exact one
        u = HALF_STEP[io]
        for b in range(B):
            e = (host(q[b, p:p + T]), host(k[b, :p + T]), host(v[b, :p + T]), window, sinks, float(np.float32(D ** -0.5)))
            assert (a[b].cpu().numpy() <= 2 * oracle.attention_bound(*e, u, u)[0]).all(), (p, T)
        p += T
        lens += T
    assert p == L


def test_strides_and_captured_steps(ops):
    # slices of a projection's rows and of a cache of keys and values side by
    # side; a captured step replayed as the lengths move
    r = np.random.default_rng(4)
    B, Hq, Hk, D, window, sinks, capacity = 3, 8, 2, 64, 1030, 2, 1034
    kv = torch.zeros((B, capacity, 2 * Hk, D), dtype=torch.bfloat16, device="cuda")
    kc, vc = kv[:, :, :Hk], kv[:, :, Hk:]
    plain = [torch.zeros((B, capacity, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qkv = draw(r, (B, 1, Hq + 2 * Hk, D), "bf16")
    lens = torch.tensor([0, 1000, 1033], device="cuda")
    see = {"window": window, "sinks": sinks}

    def step():
        return ops.window_attn_decode(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:], kc, vc, lens, **see)

    step()
    torch.cuda.synchronize()
    kv.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
        lens += 1
    for i in range(6):
        qkv.copy_(draw(r, (B, 1, Hq + 2 * Hk, D), "bf16"))
        n = lens.clone()
        parts = [t.contiguous() for t in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:])]
        want = ops.window_attn_decode(*parts, *plain, n, **see)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(kc, plain[0]) and torch.equal(vc, plain[1]), i


# one block, a few splits, many; tiles of the cache that every new token sees next to tiles that some do
SPLITS = [
    (1, 8, 2, 64, 0, 0, 320, [300]), (2, 4, 1, 128, 0, 0, 400, [383, 398]), (3, 8, 2, 72, 300, 40, 500, [100, 342, 499, 777]),
    (8, 4, 4, 128, 700, 64, 800, [70, 763, 764, 1600]), (16, 4, 1, 64, 1500, 1, 1516, [1515, 5000]),
    (1, 3, 3, 32, 0, 96, 4000, [3999, 4000, 9000]), (5, 6, 3, 96, 1000, 31, 1040, [20, 30, 31, 32, 1034, 1035, 1036, 2222]),
]


@pytest.mark.parametrize("T,Hq,Hk,D,window,sinks,capacity,lens", SPLITS)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_splits_and_full_tiles(ops, io, T, Hq, Hk, D, window, sinks, capacity, lens):
    test_against_the_oracle(ops, io, T, Hq, Hk, D, window, sinks, capacity, lens)


@pytest.mark.parametrize("window", [0, 60])
def test_very_long_sequences(ops, window):
    # positions past 32 bits: what lies at the same place of the ring is the same
    r = np.random.default_rng(8)
    sinks, capacity, T, small = 4, 100, 5, [997, 1000, 1031, 4, 95]
    ring = capacity - sinks
    q, k, v = draw(r, (5, T, 4, 64), "bf16"), draw(r, (5, T, 2, 64), "bf16"), draw(r, (5, T, 2, 64), "bf16")
    kc, vc = draw(r, (5, capacity, 2, 64), "bf16"), draw(r, (5, capacity, 2, 64), "bf16")
    got = []
    for turns in (0, 1 << 26, 1 << 40):
        c = kc.clone(), vc.clone()
        lens = torch.tensor([n + ring * (turns if n > 200 else 0) for n in small], device="cuda")
        got.append((ops.window_attn_decode(q, k, v, *c, lens, window=window, sinks=sinks),) + c)
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("window,sinks,capacity,lens", [(60, 4, 71, [0, 30, 66, 70, 100, 1000]), (1, 0, 8, [0, 5, 8, 100]),
                                                        (0, 3, 90, [0, 2, 60, 74])])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_dropped_tokens(ops, io, window, sinks, capacity, lens):
    # 8 drafted tokens, 3 of which stay: what follows is the same as over a cache that never held the others
    print(f"dropped tokens {io} window {window} capacity {capacity}", flush=True)
    r = np.random.default_rng(9)
    B, see = len(lens), {"window": window, "sinks": sinks}
    kc, vc = draw(r, (B, capacity, 2, 64), io), draw(r, (B, capacity, 2, 64), io)
    clean = kc.clone(), vc.clone()
    draft = [draw(r, (B, 8, h, 64), io) for h in (4, 2, 2)]
    n = torch.tensor(lens, device="cuda")
    ops.window_attn_decode(*draft, kc, vc, n, **see)
    ops.window_attn_decode(*(t[:, :3].contiguous() for t in draft), *clean, n, **see)
    for T in (1, 8, 4):
        new = [draw(r, (B, T, h, 64), io) for h in (4, 2, 2)]
        n = n + (3 if T == 1 else 1)  # of the 8 one stays
        got, want = (ops.window_attn_decode(*new, *c, n, **see) for c in ((kc, vc), clean))
        assert torch.equal(got, want), T
