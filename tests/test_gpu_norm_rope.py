"""Parity of the head norms with rotation with their fp64 oracle
(oracle/attention.py, pinned in tests/test_oracle_attention_pins.py).  Needs an
MI355X.  Every output entry is held to the oracle's bound for it."""
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


def draw(rng, shape, io, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda().to(IO[io])


def within(name, got, ref, bound):
    got = host(got).reshape(ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} entries off, first {i}: {got[i]} against {ref[i]}, "
                             f"bound {np.broadcast_to(bound, ref.shape)[i]}")


def rates(R):
    return torch.exp(-torch.arange(R // 2, dtype=torch.float64) * (2 * np.log(10000.0) / max(R, 1))).float().cuda()


def flat(t):
    return host(t).reshape((-1,) + tuple(t.shape[-2:]))


def check(ops, io, q, k, gq, gk, eps, theta, pos, halves, seed):
    """Forward and backward of one call against the oracle."""
    lead = q.shape[:-2]
    at = np.broadcast_to(np.arange(lead[-1]), lead).reshape(-1) if pos is None else pos.cpu().numpy().reshape(-1)
    th = None if theta is None else host(theta)
    u = HALF_STEP[io]
    turn = dict(theta=theta, pos=pos, halves=halves)
    out = ops.qk_norm_rope_fwd(q, k, gq, gk, eps, **turn)
    for name, x, g, y in (("q", q, gq, out[0]), ("k", k, gk, out[1])):
        a = (flat(x), None if g is None else host(g), eps, th, at, halves)
        within(name, y, oracle.norm_rope(*a), oracle.norm_rope_bound(*a, u))
    r = np.random.default_rng(seed)
    dq, dk = draw(r, tuple(q.shape), io), draw(r, tuple(k.shape), io)
    grads = ops.qk_norm_rope_bwd(q, k, dq, dk, gq, gk, eps, **turn)
    assert set(grads) == {"dq", "dk", "dgain_q", "dgain_k"}
    for n, x, g, dy in (("q", q, gq, dq), ("k", k, gk, dk)):
        a = (flat(x), None if g is None else host(g), eps, th, at, halves, flat(dy))
        for name, want, bound in zip(("d" + n, "dgain_" + n), oracle.norm_rope_bwd(*a), oracle.norm_rope_bwd_bound(*a, u)):
            within(name, grads[name], want, bound)
    return out, grads, (dq, dk)


# every number of lanes per head, whole and partial vectors, partial and no
# rotation, pairs that lie within and across vectors; (D, rope_dim)
WIDTHS = [(1, 0), (2, 2), (8, 8), (30, 14), (32, 32), (33, 10), (64, 64), (76, 38), (80, 40), (96, 96), (128, 128),
          (128, 64), (192, 96), (255, 254), (256, 256)]


@pytest.mark.parametrize("D,R", WIDTHS)
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_widths(ops, io, halves, D, R):
    print(f"norm_rope {io} D {D} rope {R} halves {halves}", flush=True)
    r = np.random.default_rng(D + R)
    q, k = draw(r, (2, 9, 5, D), io, 1.5), draw(r, (2, 9, 2, D), io, 0.3)
    gq, gk = draw(r, D, "f32"), draw(r, D, "f32")
    check(ops, io, q, k, gq, gk, 1e-5, rates(R) if R else None, None, halves, 1)


@pytest.mark.parametrize("rows,Hq,Hk", [(1, 1, 1), (1, 16, 4), (3, 64, 8), (257, 6, 3), (2500, 8, 8), (9000, 3, 1)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows(ops, io, rows, Hq, Hk):
    # one token to more than one pass of the backward's blocks; no gains
    r = np.random.default_rng(rows)
    q, k = draw(r, (rows, Hq, 64), io), draw(r, (rows, Hk, 64), io)
    check(ops, io, q, k, None, None, 0.25, rates(64), None, rows % 2 == 0, 2)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_far_and_negative_positions(ops, io):
    r = np.random.default_rng(3)
    q, k = draw(r, (4, 40, 3, 64), io), draw(r, (4, 40, 1, 64), io)
    pos = torch.from_numpy(r.integers(-10 ** 9, 10 ** 9, (4, 40))).cuda()
    check(ops, io, q, k, None, None, 1e-5, rates(64), pos, False, 3)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("halves", [False, True])
def test_slices_and_in_place(ops, io, halves):
    # queries and keys as slices of one projection's rows, results over them
    r = np.random.default_rng(4)
    B, L, Hq, Hk, D = 2, 33, 4, 2, 72
    qkv = draw(r, (B, L, Hq + 2 * Hk, D), io)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:].clone()
    gq, gk, th = draw(r, D, "f32"), draw(r, D, "f32"), rates(36)
    out, grads, (dq, dk) = check(ops, io, q, k, gq, gk, 1e-5, th, None, halves, 5)
    dqkv = torch.full_like(qkv, 7.0)
    dqkv[:, :, :Hq], dqkv[:, :, Hq:Hq + Hk] = dq, dk
    sq, sk = dqkv[:, :, :Hq], dqkv[:, :, Hq:Hq + Hk]
    again = ops.qk_norm_rope_bwd(q, k, sq, sk, gq, gk, theta=th, halves=halves, dq=sq, dk=sk)
    assert all(torch.equal(again[n], grads[n]) for n in grads) and bool((dqkv[:, :, Hq + Hk:] == 7.0).all())
    a, b = ops.qk_norm_rope_fwd(q, k, gq, gk, theta=th, halves=halves, q_out=q, k_out=k)
    assert torch.equal(a, out[0]) and torch.equal(b, out[1]) and torch.equal(qkv[:, :, Hq + Hk:], v)


def test_one_operand_and_no_rows(ops):
    r = np.random.default_rng(6)
    q, k, th = draw(r, (2, 5, 3, 64), "bf16"), draw(r, (2, 5, 2, 64), "bf16"), rates(64)
    both = ops.qk_norm_rope_fwd(q, k, theta=th)
    a, none = ops.qk_norm_rope_fwd(q, None, theta=th)
    nil, b = ops.qk_norm_rope_fwd(None, k, theta=th)
    assert none is None and nil is None and torch.equal(a, both[0]) and torch.equal(b, both[1])
    grads = ops.qk_norm_rope_bwd(q, None, q, None, theta=th)
    assert set(grads) == {"dq", "dgain_q"}
    full = ops.qk_norm_rope_bwd(q, k, q, k, theta=th)
    assert torch.equal(grads["dq"], full["dq"])
    only = ops.qk_norm_rope_bwd(q, k, q, k, theta=th, want_dgain=False)
    assert set(only) == {"dq", "dk"} and torch.equal(only["dk"], full["dk"])
    empty = ops.qk_norm_rope_bwd(q[:, :0], k[:, :0], q[:, :0], k[:, :0], theta=th)
    assert empty["dq"].shape == (2, 0, 3, 64) and not bool(empty["dgain_q"].any()) and not bool(empty["dgain_k"].any())


def test_bad_heads_stay_alone(ops):
    # NaN, infinity and an all-zero head without eps touch their own head only
    r = np.random.default_rng(7)
    for io in ("bf16", "f32"):
        q, k, th = draw(r, (20, 4, 64), io), draw(r, (20, 4, 64), io), rates(64)
        ref = ops.qk_norm_rope_fwd(q, k, eps=0.0, theta=th)
        bad = q.clone()
        bad[3, 1, 5], bad[7, 0, 63], bad[11, 2] = float("nan"), float("inf"), 0.0
        got, same = ops.qk_norm_rope_fwd(bad, k, eps=0.0, theta=th)
        off = torch.zeros(20, 4, dtype=torch.bool, device="cuda")
        off[3, 1] = off[7, 0] = off[11, 2] = True
        assert torch.equal(got[~off], ref[0][~off]) and torch.equal(same, ref[1])
        assert bool(got[3, 1].isnan().all()) and bool(got[11, 2].isnan().all())
