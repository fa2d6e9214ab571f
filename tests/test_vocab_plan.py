"""The plan of the vocabulary cross entropy's matrix products (no GPU): which
columns go over from large tiles to small ones.  Large tiles run 256 at a time,
one a compute unit; small tiles take a last round that fills less than half of
the units, and no more than about that."""

import ctypes

import pytest

import collective_communication_reduction_way_amd as rr

UNITS = 256
LARGE, SMALL = 0, 1


def tail_start(c0, c1, other_tiles, tile=LARGE):
    # (rr::tail_start, internal to the library)
    f = rr.lib()._ZN2rr10tail_startEjjjNS_9VocabTileE
    f.restype, f.argtypes = ctypes.c_uint32, [ctypes.c_uint32] * 3 + [ctypes.c_int]
    return f(c0, c1, other_tiles, tile)


@pytest.mark.parametrize("other", (1, 2, 7, 8, 16, 32, 100, 200, 255, 256, 257, 274, 300, 1000, 32768))
def test_columns_of_small_tiles(other):
    for cols in (1, 64, 256, 1000, 5184, 32000, 50304, 131072, 262144):
        for c0 in (0, 1 << 18):
            cm = tail_start(c0, c0 + cols, other)
            assert c0 <= cm <= c0 + cols
            tiles = -(-cols // 256) * other
            if cm == c0 + cols:
                continue
            assert (cm - c0) % 256 == 0
            moved = tiles - (cm - c0) // 256 * other
            # a part of one round, less than half of the units, behind at least one full round
            assert moved < UNITS // 2 and tiles - moved >= UNITS, (cols, moved, tiles)
            # and what stays ends with full rounds, or all but a column's tiles of the last one
            assert (tiles - moved) % UNITS == 0 or UNITS - (tiles - moved) % UNITS < other


def test_where_the_tail_pays():
    # 2048 tokens, 50257 rows: 1576 tiles are six rounds and 40 more
    assert tail_start(0, 50304, 8) == 192 * 256
    # a last round of half the units stays, and so does less than one round
    assert tail_start(0, (UNITS + 128) * 256, 1) == (UNITS + 128) * 256
    assert tail_start(0, 100 * 256, 1) == 100 * 256
    # small tiles have no tail
    assert tail_start(0, 50304, 8, SMALL) == 50304


def test_many_tokens():
    """70000 tokens are 274 tiles a column of the vocabulary, more than a round: 18
    tiles of the last round are no column of their own."""
    assert tail_start(0, 256, 274) == 256
    for cols in (256 * k for k in (2, 3, 14, 15, 21)):
        cm = tail_start(0, cols, 274)
        assert (cols - cm) // 256 * 274 < UNITS // 2
