"""The forms that the products' planner picks, one small product for each, on the
host: a change of the planner's costs that moves a size to another form shows
here, and tests/test_gpu_block_forms.py, which runs these products, does not
lose the form silently.
"""
import ctypes

import pytest

# kind, io type, rows, d_in, d_out (of the product: rows x d_in -> d_out; gated:
# twice as many rows of W), tile, how its tiles are cut ("whole": none of them,
# "split": all over k, "mixed": whole ones and split ones in one launch), and
# for the smaller tiles whether a block is alone on its CU
FORMS = [
    ("dW", "f32", 768, 4952, 1888, 128, "mixed", False),
    ("dW", "f32", 3474, 2474, 608, 128, "split", False),
    ("dW", "f32", 1234, 200, 4137, 128, "split", True),
    ("dW", "f32", 354, 1532, 4851, 128, "whole", False),
    ("dW", "f32", 358, 3912, 800, 128, "whole", True),
    ("dW", "f32", 427, 4808, 4056, 256, "mixed"),
    ("dW", "f32", 7334, 216, 2776, 256, "split"),
    ("dW", "f32", 71, 3560, 4256, 256, "whole"),
    ("dW", "f32", 491, 1731, 1212, 64, "mixed", False),
    ("dW", "f32", 937, 8, 5632, 64, "split", False),
    ("dW", "f32", 417, 8, 8, 64, "split", True),
    ("dW", "f32", 1, 4112, 200, 64, "whole", False),
    ("dW", "f32", 1, 8, 8, 64, "whole", True),
    ("dx", "f32", 9384, 976, 816, 128, "mixed", False),
    ("dx", "f32", 9109, 75, 5756, 128, "split", False),
    ("dx", "f32", 8246, 80, 1456, 128, "split", True),
    ("dx", "f32", 10376, 664, 376, 128, "whole", False),
    ("dx", "f32", 10450, 280, 368, 128, "whole", True),
    ("dx", "f32", 16010, 1280, 361, 256, "mixed"),
    ("dx", "f32", 202, 4110, 4353, 256, "split"),
    ("dx", "f32", 5295, 2773, 73, 256, "whole"),
    ("dx", "f32", 8649, 220, 466, 64, "mixed", False),
    ("dx", "f32", 1, 4383, 1739, 64, "split", False),
    ("dx", "f32", 1, 8, 440, 64, "split", True),
    ("dx", "f32", 8400, 72, 8, 64, "whole", False),
    ("dx", "f32", 1, 8, 8, 64, "whole", True),
    ("gated", "f32", 11209, 2910, 325, 128, "mixed", False),
    ("gated", "f32", 15572, 1800, 208, 128, "whole", False),
    ("gated", "f32", 3461, 1720, 392, 128, "whole", True),
    ("gated", "f32", 14879, 568, 584, 256, "mixed"),
    ("gated", "f32", 4254, 4633, 72, 256, "split"),
    ("gated", "f32", 15074, 107, 466, 256, "whole"),
    ("gated", "f32", 523, 301, 3716, 64, "mixed", False),
    ("gated", "f32", 5484, 616, 8, 64, "split", False),
    ("gated", "f32", 65, 359, 8, 64, "split", True),
    ("gated", "f32", 8961, 9, 71, 64, "whole", False),
    ("gated", "f32", 67, 8, 8, 64, "whole", True),
    ("linear", "f32", 2773, 672, 3440, 128, "mixed", False),
    ("linear", "f32", 12557, 4362, 80, 128, "split", False),
    ("linear", "f32", 10273, 1104, 72, 128, "split", True),
    ("linear", "f32", 1237, 377, 5898, 128, "whole", False),
    ("linear", "f32", 10151, 432, 258, 128, "whole", True),
    ("linear", "f32", 9517, 360, 1976, 256, "mixed"),
    ("linear", "f32", 252, 4909, 4177, 256, "split"),
    ("linear", "f32", 9176, 72, 1725, 256, "whole"),
    ("linear", "f32", 11149, 535, 132, 64, "mixed", False),
    ("linear", "f32", 6395, 776, 8, 64, "split", False),
    ("linear", "f32", 65, 600, 8, 64, "split", True),
    ("linear", "f32", 8698, 8, 80, 64, "whole", False),
    ("linear", "f32", 65, 8, 8, 64, "whole", True),
    ("dW", "bf16", 8156, 188, 5916, 128, "split", False),
    ("dW", "bf16", 3239, 66, 3410, 128, "split", True),
    ("dW", "bf16", 1, 2408, 2592, 128, "whole", False),
    ("dW", "bf16", 1, 1368, 2184, 128, "whole", True),
    ("dW", "bf16", 961, 3392, 4952, 256, "mixed"),
    ("dW", "bf16", 9015, 152, 5632, 256, "split"),
    ("dW", "bf16", 67, 4200, 3176, 256, "whole"),
    ("dW", "bf16", 3355, 4416, 8, 64, "split", False),
    ("dW", "bf16", 1552, 8, 8, 64, "split", True),
    ("dW", "bf16", 1, 3505, 259, 64, "whole", False),
    ("dW", "bf16", 1, 8, 8, 64, "whole", True),
    ("dx", "bf16", 1177, 1783, 4817, 128, "split", False),
    ("dx", "bf16", 2779, 65, 3667, 128, "split", True),
    ("dx", "bf16", 7093, 856, 8, 128, "whole", False),
    ("dx", "bf16", 7003, 392, 8, 128, "whole", True),
    ("dx", "bf16", 9718, 1784, 712, 256, "mixed"),
    ("dx", "bf16", 8817, 211, 5275, 256, "split"),
    ("dx", "bf16", 8555, 1556, 65, 256, "whole"),
    ("dx", "bf16", 1, 2696, 4808, 64, "split", False),
    ("dx", "bf16", 1, 8, 1416, 64, "split", True),
    ("dx", "bf16", 9884, 72, 8, 64, "whole", False),
    ("dx", "bf16", 1, 8, 8, 64, "whole", True),
    ("gated", "bf16", 5502, 4672, 153, 128, "split", False),
    ("gated", "bf16", 4258, 2344, 8, 128, "split", True),
    ("gated", "bf16", 12584, 130, 218, 128, "whole", False),
    ("gated", "bf16", 8329, 152, 72, 128, "whole", True),
    ("gated", "bf16", 5915, 942, 1345, 256, "mixed"),
    ("gated", "bf16", 1614, 3272, 1224, 256, "split"),
    ("gated", "bf16", 10318, 72, 592, 256, "whole"),
    ("gated", "bf16", 131, 1581, 1851, 64, "split", False),
    ("gated", "bf16", 71, 974, 8, 64, "split", True),
    ("gated", "bf16", 8649, 8, 80, 64, "whole", False),
    ("gated", "bf16", 65, 8, 8, 64, "whole", True),
    ("linear", "bf16", 1576, 4795, 1400, 128, "split", False),
    ("linear", "bf16", 65, 3552, 3384, 128, "split", True),
    ("linear", "bf16", 3333, 8, 1853, 128, "whole", False),
    ("linear", "bf16", 10414, 8, 264, 128, "whole", True),
    ("linear", "bf16", 4410, 687, 3727, 256, "mixed"),
    ("linear", "bf16", 917, 3032, 4360, 256, "split"),
    ("linear", "bf16", 11450, 65, 1055, 256, "whole"),
    ("linear", "bf16", 4244, 3040, 8, 64, "split", False),
    ("linear", "bf16", 68, 1416, 8, 64, "split", True),
    ("linear", "bf16", 193, 8, 4103, 64, "whole", False),
    ("linear", "bf16", 65, 8, 8, 64, "whole", True),
]
# products of ordinary sizes on the widest tiles, inside the matrix and ragged
ORDINARY = [
    ("linear", "bf16", 4352, 2048, 4352, 256, "mixed"),
    ("linear", "bf16", 4200, 3000, 4200, 256, "mixed"),
    ("gated", "bf16", 4352, 2048, 2176, 256, "mixed"),
    ("dx", "bf16", 4352, 4352, 4096, 256, "mixed"),
    ("dW", "bf16", 4096, 4352, 4352, 256, "mixed"),
    ("dW", "bf16", 2048, 4096, 4096, 256, "whole"),
    ("dx", "bf16", 4096, 4096, 1000, 256, "whole"),
    ("linear", "f32", 8192, 1024, 4096, 256, "whole"),
    ("linear", "f32", 8192, 1024, 2200, 256, "mixed"),
    ("gated", "f32", 8192, 512, 1024, 256, "whole"),
]
ALL = FORMS + ORDINARY
IDS = ["-".join(str(v) for v in c) for c in ALL]
EPILOGUE = {"dx": 0, "dW": 0, "linear": 1, "gated": 2}
RESIDENT = {256: 256, 128: 512, 64: 512}  # blocks on the chip


@pytest.fixture(scope="module")
def plan():
    import os
    from state_space_sequence_03_amd import ops
    if not os.path.exists(ops.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    query = ops.lib().m3_product_plan
    query.argtypes = [ctypes.c_int, ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int64)]
    query.restype = None

    def plan(kind, io, rows, d_in, d_out):
        """tile, tiles, whole ones, parts of each other tile"""
        out = (ctypes.c_int64 * 4)()
        m, n, k = {"dx": (rows, d_in, d_out), "dW": (d_out, d_in, rows)}.get(kind, (rows, d_out, d_in))
        query(io == "bf16", EPILOGUE[kind], m, n, k, out)
        return tuple(out)

    return plan


def form(plan, kind, io, rows, d_in, d_out):
    tile, tiles, whole, parts = plan(kind, io, rows, d_in, d_out)
    if tile == 0:
        return (0,)
    cut = "whole" if parts == 1 else "split" if whole == 0 else "mixed"
    if tile == 256:
        return tile, cut
    items = tiles if parts == 1 else whole + (tiles - whole) * parts
    return tile, cut, items <= 256


@pytest.mark.parametrize("case", ALL, ids=IDS)
def test_plan(plan, case):
    assert form(plan, *case[:5]) == case[5:]


def test_every_form_is_listed_once():
    assert len({(c[0], c[1]) + c[5:] for c in FORMS}) == len(FORMS)
    for kind in EPILOGUE:
        for io in ("bf16", "f32"):
            listed = {c[5:7] for c in FORMS if c[:2] == (kind, io)}
            assert {(256, cut) for cut in ("whole", "split", "mixed")} <= listed
            assert {(tile, cut) for tile in (128, 64) for cut in ("whole", "split")} - listed <= {(128, "split")}


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_parts_cover_a_plan(plan, io):
    # tiles cover the result; only the last, partial round of tiles is ever split
    for rows in (1, 65, 777, 4097, 20000):
        for d_in, d_out in ((8, 8), (1000, 1531), (2048, 5632), (4110, 96)):
            for kind in EPILOGUE:
                tile, tiles, whole, parts = plan(kind, io, rows, d_in, d_out)
                if tile == 0:
                    assert kind in ("linear", "gated") and rows <= 64
                    continue
                m, n = {"dx": (rows, d_in), "dW": (d_out, d_in)}.get(kind, (rows, d_out))
                across = tile // 2 if kind == "gated" and tile > 64 else tile
                assert tiles == -(-m // tile) * -(-n // across)
                assert 0 <= whole <= tiles and 1 <= parts <= 64
                assert whole == tiles if parts == 1 else whole % RESIDENT[tile] == 0 and whole < tiles
