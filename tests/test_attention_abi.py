"""Host-side checks of the attention layer's entry points (no GPU, nothing is
launched): the documented refusals, workspace sizes and empty calls."""
import ctypes
import os

import pytest

FAKE = 0x7F0000000000  # aligned fake device address (never touched)


@pytest.fixture(scope="module")
def L():
    from state_space_sequence_03_amd import ops
    if not os.path.exists(ops.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return ops


def made(struct, base, kw):
    d = struct()
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


def turn(L, **kw):
    return made(L.NormRopeDims, dict(rows=6, seqlen=3, q_heads=4, k_heads=2, head_dim=64, rope_dim=64, io_dtype=L.M3_BF16),
                kw)


def attn(L, **kw):
    return made(L.AttnDims, dict(batch=2, q_len=5, kv_len=7, q_heads=4, kv_heads=2, head_dim=64, window=3, sinks=1,
                                 scale=0.125, io_dtype=L.M3_BF16), kw)


def step(L, **kw):
    return made(L.AttnDecodeDims, dict(batch=2, tokens=2, capacity=40, q_heads=4, kv_heads=2, head_dim=64, window=30,
                                       sinks=1, scale=0.125, io_dtype=L.M3_BF16), kw)


TURN = ("q", "k", "gain_q", "gain_k", "eps", "theta", "pos", "q_out", "k_out")
TURN_BWD = ("q", "k", "dq_out", "dk_out", "gain_q", "gain_k", "eps", "theta", "pos", "dq", "dk", "dgain_q", "dgain_k")
FWD = ("q", "k", "v", "starts", "o", "lse")
BWD = ("q", "k", "v", "o", "lse", "dout", "starts", "dq", "dk", "dv")
STEP = ("q", "k", "v", "k_cache", "v_cache", "lens", "o")
NO_WORKSPACE = ("qk_norm_rope_fwd", "window_attn_fwd")


def call(L, fn, names, dims, ws=FAKE, ws_bytes=1 << 60, **over):
    args = [over.get(n, 1e-5 if n == "eps" else FAKE) for n in names]
    tail = [None] if fn in NO_WORKSPACE else [ws, ws_bytes, None]
    return getattr(L.lib(), "mamba3_" + fn)(None if dims is None else ctypes.byref(dims), *args, *tail)


@pytest.mark.parametrize("fn,names", [("qk_norm_rope_fwd", TURN), ("qk_norm_rope_bwd", TURN_BWD)])
def test_norm_rope_refusals(L, fn, names):
    go = lambda ws=FAKE, over={}, **kw: call(L, fn, names, turn(L, **kw), ws, **over)
    assert call(L, fn, names, None) == L.M3_ERR_NULL
    for bad in (dict(rows=-1), dict(seqlen=-1), dict(q_heads=-1), dict(k_heads=-1), dict(head_dim=0), dict(rope_dim=-2),
                dict(rope_dim=31), dict(rope_dim=66), dict(q_stride=255), dict(k_stride=127), dict(q_out_stride=255),
                dict(k_out_stride=127)):
        assert go(**bad) == L.M3_ERR_SHAPE, bad
    for bad in (dict(rows=1 << 24), dict(head_dim=258, rope_dim=0), dict(io_dtype=2), dict(flags=1),
                dict(q_heads=(1 << 20) // 64 + 1), dict(q_stride=(1 << 20) + 1), dict(k_out_stride=(1 << 20) + 1)):
        assert go(**bad) == L.M3_ERR_UNSUPPORTED, bad
    for eps in (-1.0, float("nan"), float("inf")):
        assert go(over={"eps": eps}) == L.M3_ERR_UNSUPPORTED
    need = ["q", "k", "theta"] + (["q_out", "k_out"] if fn.endswith("fwd") else ["dq_out", "dk_out", "dq", "dk"])
    for n in need:
        assert go(over={n: None}) == L.M3_ERR_NULL, n
        assert go(over={n: FAKE + (2 if n == "theta" else 1)}) == L.M3_ERR_ALIGN, n
    for n, off in (("gain_q", 2), ("gain_k", 2), ("pos", 4)):
        assert go(over={n: FAKE + off}) == L.M3_ERR_ALIGN, n
    assert go(io_dtype=L.M3_F32, over={"q": FAKE + 2}) == L.M3_ERR_ALIGN
    # no rows: nothing is read or asked for
    none = {n: None for n in names if n != "eps"}
    assert go(ws=None, rows=0, over=none) == L.M3_OK
    assert go(ws=None, q_heads=0, k_heads=0, rope_dim=0, over=none) == L.M3_OK
    if fn.endswith("bwd"):
        for bad in (dict(dq_stride=255), dict(dk_stride=127)):
            assert go(**bad) == L.M3_ERR_SHAPE, bad
        size = L.qk_norm_rope_bwd_workspace_size(turn(L))
        assert size > 0 and size % (8 * 64) == 0
        assert call(L, fn, names, turn(L), ws_bytes=size - 1) == L.M3_ERR_WORKSPACE
        assert go(ws=None) == L.M3_ERR_WORKSPACE
        assert L.qk_norm_rope_bwd_workspace_size(turn(L, rope_dim=3)) == 0
        assert L.qk_norm_rope_bwd_workspace_size(turn(L, rows=0)) == 0


@pytest.mark.parametrize("fn,names", [("window_attn_fwd", FWD), ("window_attn_bwd", BWD)])
def test_attention_refusals(L, fn, names):
    go = lambda ws=FAKE, over={}, **kw: call(L, fn, names, attn(L, **kw), ws, **over)
    assert call(L, fn, names, None) == L.M3_ERR_NULL
    packed = dict(flags=L.M3_FLAG_PACKED, rows=9)
    for bad in (dict(batch=-1), dict(q_len=-1), dict(kv_len=-1), dict(q_heads=0), dict(kv_heads=0), dict(kv_heads=3),
                dict(head_dim=0), dict(window=-1), dict(sinks=-1), dict(q_stride=248), dict(k_stride=120),
                dict(v_stride=120), dict(o_stride=248), dict(kv_rows=6), dict(packed, rows=-1)):
        assert go(**bad) == L.M3_ERR_SHAPE, bad
    for bad in (dict(head_dim=136), dict(head_dim=60), dict(io_dtype=7), dict(flags=1), dict(reserved=1), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_len=1 << 24),
                dict(kv_len=1 << 24), dict(batch=1 << 24), dict(batch=1 << 13, q_len=1 << 12, kv_len=1),
                dict(batch=1 << 20, q_heads=64), dict(q_heads=1 << 15, kv_heads=1 << 15), dict(q_stride=(1 << 20) + 8),
                dict(packed, rows=1 << 24)):
        assert go(**bad) == L.M3_ERR_UNSUPPORTED, bad
    for bad in (dict(q_stride=260), dict(k_stride=132), dict(v_stride=132), dict(o_stride=260),
                dict(io_dtype=L.M3_F32, q_stride=258)):
        assert go(**bad) == L.M3_ERR_ALIGN, bad
    need = ["q", "k", "v", "o"] + (["lse", "dout"] if fn.endswith("bwd") else [])
    for n in need:
        assert go(over={n: None}) == L.M3_ERR_NULL, n
    assert go(over={"starts": None}, **packed) == L.M3_ERR_NULL
    for n in names:
        off = {"lse": 2, "starts": 4}.get(n, 8)
        assert go(over={n: FAKE + off}, **(packed if n == "starts" else {})) == L.M3_ERR_ALIGN, n
    # no sequences: nothing is read
    none = {n: None for n in names}
    assert go(ws=None, batch=0, over=none) == L.M3_OK
    assert go(ws=None, batch=0, over=none, **{**packed, "rows": 0}) == L.M3_OK
    if fn.endswith("bwd"):
        for bad in (dict(do_stride=248), dict(dq_stride=248), dict(dk_stride=120), dict(dv_stride=120)):
            assert go(**bad) == L.M3_ERR_SHAPE, bad
        assert go(dv_stride=132) == L.M3_ERR_ALIGN
        size = L.window_attn_bwd_workspace_size(attn(L))
        assert size >= 2 * 4 * 4 * 10
        assert call(L, fn, names, attn(L), ws_bytes=size - 1) == L.M3_ERR_WORKSPACE
        assert go(ws=None) == L.M3_ERR_WORKSPACE
        # no gradient asked for: done after the checks
        assert go(ws=None, over={"dq": None, "dk": None, "dv": None}) == L.M3_OK
        assert L.window_attn_bwd_workspace_size(attn(L, head_dim=12)) == 0
    else:
        assert go(ws=None, q_len=0, over=none) == L.M3_OK


def test_backward_workspace_stays_small(L):
    # two statistics per query and head, and the sinks' pieces: bounded whatever the window and the sinks
    for kw in (dict(batch=8, q_len=4096, kv_len=4096, window=1024, sinks=4), dict(batch=1, q_len=1 << 20, kv_len=1 << 20, window=16, sinks=4),
               dict(batch=1, q_len=65536, kv_len=65536, window=16, sinks=20000), dict(batch=4096, q_len=300, kv_len=300, window=16, sinks=16),
               dict(flags=L.M3_FLAG_PACKED, batch=5000, rows=1 << 20, window=64, sinks=130)):
        d = attn(L, q_heads=32, kv_heads=8, head_dim=128, **kw)
        rows = kw.get("rows") or kw["batch"] * kw["q_len"]
        assert L.window_attn_bwd_workspace_size(d) <= 8 * 32 * rows + 512 + 16384 * 8 * 32 * 128 * 4, kw


def test_decode_refusals(L):
    fn, names = "window_attn_decode", STEP
    go = lambda ws=FAKE, over={}, **kw: call(L, fn, names, step(L, **kw), ws, **over)
    assert call(L, fn, names, None) == L.M3_ERR_NULL
    for bad in (dict(batch=-1), dict(tokens=0), dict(capacity=0), dict(q_heads=0), dict(kv_heads=3), dict(head_dim=-8),
                dict(window=-1), dict(sinks=-1), dict(sinks=40), dict(sinks=10), dict(window=39), dict(window=0, sinks=39),
                dict(q_stride=248), dict(k_stride=120), dict(v_stride=120), dict(o_stride=248), dict(k_cache_stride=120),
                dict(v_cache_stride=120)):
        assert go(**bad) == L.M3_ERR_SHAPE, bad
    for bad in (dict(tokens=17), dict(capacity=(1 << 30) + 1), dict(head_dim=136), dict(head_dim=4), dict(io_dtype=2),
                dict(flags=L.M3_FLAG_PACKED), dict(reserved=1), dict(scale=0.0), dict(batch=1 << 24),
                dict(batch=1 << 23, q_heads=8, kv_heads=8), dict(k_cache_stride=(1 << 20) + 8)):
        assert go(**bad) == L.M3_ERR_UNSUPPORTED, bad
    for bad in (dict(q_stride=260), dict(k_stride=132), dict(v_cache_stride=132)):
        assert go(**bad) == L.M3_ERR_ALIGN, bad
    for n in names:
        assert go(over={n: None}) == L.M3_ERR_NULL, n
        assert go(over={n: FAKE + (4 if n == "lens" else 8)}) == L.M3_ERR_ALIGN, n
    assert go(ws=None, batch=0, over={n: None for n in names}) == L.M3_OK
    # what fits: a window that fills the ring exactly; a long cache's parts need room
    long = dict(batch=1, capacity=100000, window=0, sinks=0)
    need = L.window_attn_decode_workspace_size(step(L, **long))
    assert need > 0 and call(L, fn, names, step(L, **long), ws_bytes=need - 1) == L.M3_ERR_WORKSPACE
    assert go(ws=None, **long) == L.M3_ERR_WORKSPACE
    assert L.window_attn_decode_workspace_size(step(L, window=38)) == L.window_attn_decode_workspace_size(step(L)) == 0
    assert L.window_attn_decode_workspace_size(step(L, window=39)) == 0  # refused
    # ... however long the cache: its window counts
    assert L.window_attn_decode_workspace_size(step(L, capacity=1 << 20)) == 0


def test_dims_match_the_header(L, tmp_path):
    # sizes and offsets of the structures as a C compiler lays them out
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, names = tmp_path / "p.c", {"m3_norm_rope_dims": L.NormRopeDims, "m3_attn_dims": L.AttnDims,
                                   "m3_attn_decode_dims": L.AttnDecodeDims}
    lines = [f'printf("%zu\\n", sizeof({n}));' +
             "".join(f'printf("%zu\\n", offsetof({n}, {f}));' for f, _ in s._fields_) for n, s in names.items()]
    src.write_text('#include <stdio.h>\n#include "mamba3_ssm.h"\nint main(void) {' + "\n".join(lines) + " return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "p")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "p")], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in names.values():
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want


def test_scales_that_leave_the_range(L):
    # the kernels take scores times scale log2(e): a scale whose product with it is infinite made NaN of scores of 0
    for fn, names, dims in (("window_attn_fwd", FWD, attn), ("window_attn_bwd", BWD, attn), ("window_attn_decode", STEP, step)):
        for scale in (2.36e38, 2.9e38, 3.0e38):
            assert call(L, fn, names, dims(L, scale=scale)) == L.M3_ERR_UNSUPPORTED, (fn, scale)
        for scale in (1e-40, 2.35e38):
            assert call(L, fn, names, dims(L, scale=scale, batch=0)) == L.M3_OK, (fn, scale)


def test_backward_workspace_of_packed_sequences(L):
    # the pieces that there can be, and no more: those of equal lengths and one for every sequence; 8192 at most
    def units(**kw):
        d = attn(L, q_heads=64, kv_heads=8, head_dim=128, **kw)
        rows = kw.get("rows") or kw["batch"] * kw["q_len"]
        return (L.window_attn_bwd_workspace_size(d) - 2 * ((4 * 64 * rows + 255) // 256 * 256)) / (8 * 32 * 128 * 4)

    packed = dict(flags=L.M3_FLAG_PACKED, window=16, sinks=130)
    whole = units(batch=1, q_len=16384, kv_len=16384, window=16, sinks=130)
    assert whole == 64 * 5 * 8
    for batch in (1, 2, 21, 64, 5000):
        assert units(batch=batch, rows=16384, **packed) == whole + min(batch, 64) * 5 * 8, batch
    for batch in (1, 5000):
        for rows in (65536, 1 << 18):
            for sinks in (1, 130, 512, 3000):
                assert units(batch=batch, rows=rows, **{**packed, "sinks": sinks}) <= 8192, (batch, rows, sinks)


def test_documented_limits(L):
    # each limit and the next size; nothing is launched: an accepted call ends at a null pointer, or has no queries
    N = (1 << 24) - 1

    def fwd(**kw):
        return call(L, "window_attn_fwd", FWD, attn(L, **{**dict(head_dim=8, window=0, sinks=0), **kw}), q=None)

    def bwd(**kw):
        return call(L, "window_attn_bwd", BWD, attn(L, **{**dict(head_dim=8, window=0, sinks=0), **kw}), q=None, k=None)

    one = dict(q_heads=1, kv_heads=1)
    tiles = dict(batch=N // 255, q_len=1, kv_len=0)  # 255 divides 2^24 - 1
    keys = dict(batch=(N - 32768) // 255, q_len=0, kv_len=1)
    packed = dict(one, flags=L.M3_FLAG_PACKED, rows=N)
    for go in (fwd, bwd):
        fits = L.M3_ERR_NULL
        none = L.M3_OK if go is fwd else L.M3_ERR_NULL
        assert go(**tiles, q_heads=255, kv_heads=255) == fits
        assert go(**tiles, q_heads=256, kv_heads=256) == L.M3_ERR_UNSUPPORTED
        assert go(**keys, q_heads=255, kv_heads=255) == none
        assert go(**{**keys, "batch": keys["batch"] + 1}, q_heads=255, kv_heads=255) == L.M3_ERR_UNSUPPORTED
        assert go(**one, batch=1, q_len=N, kv_len=N) == fits
        for bad in (dict(batch=2, q_len=1 << 23, kv_len=1), dict(batch=2, q_len=1, kv_len=1 << 23)):
            assert go(**one, **bad) == L.M3_ERR_UNSUPPORTED, bad
        assert go(**one, batch=1, q_len=1, kv_len=1, kv_rows=1 << 40) == fits
        assert go(**one, batch=1, q_len=1, kv_len=1, kv_rows=(1 << 40) + 1) == L.M3_ERR_UNSUPPORTED
        most = N - 32768 - N // 128
        assert go(**packed, batch=most) == fits
        assert go(**packed, batch=most + 1) == L.M3_ERR_UNSUPPORTED
    # the backward's statistics, sixteen heads of a token to a block
    wide = dict(flags=L.M3_FLAG_PACKED, batch=1, q_heads=32, kv_heads=4)
    assert fwd(**wide, rows=N // 2 + 1) == L.M3_ERR_NULL and bwd(**wide, rows=N // 2) == L.M3_ERR_NULL
    assert bwd(**wide, rows=N // 2 + 1) == L.M3_ERR_UNSUPPORTED
    # new tokens over a cache
    for T, status in ((L.M3_DECODE_MAX_TOKENS, L.M3_ERR_NULL), (L.M3_DECODE_MAX_TOKENS + 1, L.M3_ERR_UNSUPPORTED)):
        assert call(L, "window_attn_decode", STEP, step(L, tokens=T, capacity=100, window=30), q=None) == status
