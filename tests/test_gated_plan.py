"""The plan of the gated projections' matrix products (no GPU): the tiles, parts
and pieces that shapes take, so that the tests of the kernels know which of them they
run.  SHAPES reach the largest tiles in every use; test_gpu_gated_tiles runs them."""

import collections
import ctypes

import pytest

import collective_communication_reduction_way_amd as rr

U32, U64 = ctypes.c_uint32, ctypes.c_uint64
DTYPES = {"float32": 1, "bfloat16": 2, "float16": 3}
TILES = ("256", "128", "128x64", "128x32", "64", "few", "256x192")
FORWARD, WIDE, WEIGHTS = range(3)  # rr::GatedUse


class Shards(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p * 64), ("up", ctypes.c_void_p * 64), ("off", U32 * 65), ("rows", U32 * 64),
                ("p", ctypes.c_int32)]


class GatedPlan(ctypes.Structure):  # rr::GatedPlan, internal to the library
    _fields_ = [("sh", Shards)] + [(n, U32) for n in ("tokens", "dim", "dim_pad", "esz", "acc_ld", "piece")] + [
        ("ld", U64)] + [(n, ctypes.c_int) for n in ("forward", "hidden", "weight")] + [
        (n, U32) for n in ("splits", "weight_splits")] + [
        (n, U64) for n in ("pack_x", "pack_w", "grad", "pre", "acc", "weight_acc", "xs", "row_max", "row_exp", "scale",
                           "total")]


# forward, kept: the forward pass without and with its products kept (so is the gradient's, that computes them
# again), and the columns of its small tiles behind the large ones; hidden, weight: of the gradients
Plan = collections.namedtuple("Plan", "forward forward_tail kept kept_tail hidden splits pieces weight weight_splits "
                                      "weight_tail")


def plan_gated(p, tokens, dim, ffn, dtype, grad, pack, kept):
    f = rr.lib()._ZN2rr10plan_gatedERNS_9GatedPlanEijjj10rr_dtype_tbbb
    f.restype, f.argtypes = None, [ctypes.c_void_p, ctypes.c_int, U32, U32, U32, ctypes.c_int] + [ctypes.c_bool] * 3
    pl = GatedPlan()
    f(ctypes.byref(pl), p, tokens, dim, ffn, DTYPES[dtype], grad, pack, kept)
    return pl


def tail(c0, c1, other, steps, tile, f32, use):
    f = rr.lib()._ZN2rr10gated_tailEjjjjNS_9GatedTileEbNS_8GatedUseE
    f.restype, f.argtypes = U32, [U32] * 4 + [ctypes.c_int, ctypes.c_bool, ctypes.c_int]
    return c1 - f(c0, c1, other, steps, tile, f32, use)


def plan(p, tokens, dim, ffn, dtype):
    """What a call on aligned buffers takes; rows of whole 16 bytes are not copied."""
    f32 = dtype == "float32"
    pack = dim * (4 if f32 else 2) % 16 != 0
    one, two, grad = (plan_gated(p, tokens, dim, ffn, dtype, g, pack, k)
                      for g, k in ((False, False), (False, True), (True, False)))
    # what is computed again is what was kept; and the products given change nothing but the workspace
    given = plan_gated(p, tokens, dim, ffn, dtype, True, pack, True)
    assert grad.forward == two.forward
    assert all(getattr(grad, n) == getattr(given, n) for n in ("hidden", "weight", "splits", "weight_splits", "piece"))
    cols = 2 * one.sh.off[p]
    assert cols == one.ld

    def tails(pl, use):
        starts = range(0, cols, 2 * pl.piece)
        return max(tail(c, min(cols, c + 2 * pl.piece), tokens, -(-dim // 64), pl.forward, f32, use) for c in starts)

    return Plan(TILES[one.forward], tails(one, FORWARD), TILES[two.forward], tails(two, WIDE), TILES[grad.hidden],
                grad.splits, -(-cols // (2 * grad.piece)), TILES[grad.weight], grad.weight_splits,
                tail(0, cols, dim, -(-tokens // 64), grad.weight, f32, WEIGHTS))


SHAPES = {  # (p, tokens, dim, ffn): plans in float32 and in 16-bit types
    (3, 7953, 32, 894): (Plan("256", 0, "256", 0, "128x64", 4, 1, "128x64", 8, 0),
        Plan("128", 0, "128", 0, "128", 4, 1, "128", 15, 0)),
    (3, 8480, 32, 771): (Plan("256", 128, "256", 128, "128x64", 3, 1, "128x64", 8, 0),
        Plan("128", 0, "128", 0, "128", 3, 1, "128", 16, 0)),
    (1, 784, 465, 18407): (Plan("256", 2048, "256", 2048, "128x64", 9, 2, "128x64", 1, 0),
        Plan("128", 0, "128", 0, "128", 9, 1, "256", 1, 4096)),
    (2, 4374, 32, 18497): (Plan("256", 768, "256", 768, "256", 14, 1, "128x64", 1, 0),
        Plan("128", 0, "128", 0, "256", 14, 1, "128", 1, 0)),
    (3, 2115, 272, 12258): (Plan("256", 2816, "256", 2816, "128x64", 5, 1, "256", 1, 0),
        Plan("128", 0, "128", 0, "128", 5, 1, "128", 1, 0)),
    (1, 2060, 280, 16635): (Plan("256", 0, "256", 0, "128x64", 5, 1, "256", 1, 512),
        Plan("128", 0, "128", 0, "128", 5, 1, "128", 1, 0)),
    (1, 2360, 769, 16511): (Plan("256", 0, "256", 0, "256", 6, 2, "256", 1, 256),
        Plan("128", 0, "128", 0, "256", 6, 1, "128", 1, 0)),
    (2, 8300, 2568, 900): (Plan("256", 256, "256", 256, "256", 1, 1, "128x64", 1, 0),
        Plan("256", 256, "256", 256, "256", 1, 1, "128", 1, 0)),
    (2, 8200, 2049, 1090): (Plan("256", 512, "256", 512, "256", 1, 1, "128x64", 1, 0),
        Plan("128", 0, "128", 0, "256", 1, 1, "128", 1, 0)),
    (2, 1327, 193, 4458): (Plan("128x64", 0, "128x64", 0, "128x64", 12, 1, "128x64", 1, 0),
        Plan("256x192", 0, "256x192", 0, "128", 11, 1, "128", 1, 0)),
    (2, 752, 1089, 15845): (Plan("128x64", 0, "128x64", 0, "128x64", 9, 3, "128x64", 1, 0),
        Plan("256x192", 0, "256x192", 0, "128", 4, 2, "128", 1, 0)),
    (3, 9147, 2056, 625): (Plan("128x64", 0, "128x64", 0, "128x64", 1, 1, "128x64", 1, 0),
        Plan("256", 0, "256", 0, "128", 1, 1, "128", 1, 0)),
    (2, 912, 2153, 13067): (Plan("128x64", 0, "128x64", 0, "128x64", 2, 4, "128x64", 1, 0),
        Plan("256", 0, "256", 0, "128", 3, 2, "128", 1, 0)),
    (3, 6179, 2072, 1235): (Plan("256", 128, "256", 128, "128x64", 2, 1, "128x64", 1, 0),
        Plan("256", 128, "256", 128, "128", 1, 1, "128", 1, 0)),
    (1, 1677, 2121, 9698): (Plan("128x64", 0, "128x64", 0, "128x64", 1, 3, "128x64", 1, 0),
        Plan("256", 512, "256", 512, "128", 1, 2, "256", 1, 0)),
    (1, 738, 392, 13589): (Plan("256", 5504, "256", 5504, "128x64", 10, 1, "128x64", 1, 0),
        Plan("128", 0, "128", 0, "128", 10, 1, "256", 1, 0)),
    (1, 763, 393, 17384): (Plan("256", 0, "256", 0, "128x64", 21, 1, "128x64", 1, 0),
        Plan("128", 0, "128", 0, "128", 10, 1, "256", 1, 2048)),
    (2, 1289, 1345, 18386): (Plan("256", 1536, "256", 1536, "128x64", 2, 3, "128x64", 1, 0),
        Plan("256x192", 0, "256x192", 0, "256", 7, 2, "256", 1, 4096)),
    (3, 8364, 712, 605): (Plan("128x64", 0, "128x64", 0, "128x64", 3, 1, "128x64", 1, 0),
        Plan("256", 0, "128", 0, "128", 1, 1, "128", 3, 0)),
    (3, 7427, 641, 963): (Plan("256", 256, "256", 256, "128x64", 2, 1, "128x64", 1, 0),
        Plan("256", 256, "128", 0, "128", 1, 1, "128", 2, 0)),
}


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_tiles_of_shapes(shape):
    f32, b16 = SHAPES[shape]
    assert plan(*shape, "float32") == f32
    assert plan(*shape, "bfloat16") == b16 and plan(*shape, "float16") == b16


def test_every_use_of_the_large_tiles_is_reached():
    for i, large in enumerate((("256",), ("256", "256x192"))):
        plans = [both[i] for both in SHAPES.values()]
        for tile in large:
            for pieces in (False, True):
                assert any(pl.kept == tile and (pl.pieces > 1) == pieces for pl in plans), (tile, pieces)
        for some in (False, True):
            assert any(pl.forward == "256" and (pl.forward_tail > 0) == some for pl in plans)
            assert any(pl.kept == "256" and (pl.kept_tail > 0) == some for pl in plans)
            assert any(pl.weight == "256" and (pl.weight_tail > 0) == some for pl in plans)
            assert any(pl.hidden == "256" and (pl.splits > 1) == some and pl.pieces == 1 for pl in plans)
        assert any(pl.hidden == "256" and pl.pieces > 1 for pl in plans)


def test_tails_are_parts_of_a_round():
    for dtype in DTYPES:
        f32 = dtype == "float32"
        for other in (1, 300, 2048, 4096, 5001, 70000):
            for cols in (256, 5120, 22016, 32768, 1 << 20):
                for steps in (1, 16, 64, 300):
                    for use in (FORWARD, WIDE, WEIGHTS):
                        moved = tail(0, cols, other, steps, 0, f32, use)
                        across = -(-other // 256)
                        tiles = moved // 256 * across
                        # what does not fill a round, and what a column of tiles has of the round before
                        assert moved % 256 == 0 and tiles < (128 if f32 else 256 + across)
                        if moved:
                            assert (cols - moved) // 256 * across > 256 - across
                        for tile in (1, 2, 6):
                            assert tail(0, cols, other, steps, tile, f32, use) == 0
