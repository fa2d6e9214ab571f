"""Pins of the oracle of the training operators (no GPU): the generator against
its authors' published vectors, dropout against hand-made cases, the cross
entropy against closed forms and differences."""

import math

import numpy as np
import pytest

from oracle import training as TR


@pytest.mark.parametrize("counter,key,want", [
    # the known answers published with the generator
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(int(v) for v in TR.philox4x32(np.array(counter, dtype=np.uint64), key)) == want


def test_mask_is_a_function_of_the_index():
    full = TR.dropout_keep(10007, 0.3, 2 ** 63 + 5, 2 ** 40 + 9)
    assert np.array_equal(TR.dropout_keep(77, 0.3, 2 ** 63 + 5, 2 ** 40 + 9, start=1003), full[1003:1080])
    assert abs(full.mean() - 0.7) < 5 * math.sqrt(0.21 / 10007)
    assert TR.dropout_keep(100, 0.0, 1, 2).all()
    far = 4 * (2 ** 32 - 1)  # block numbers that pass 32 bits
    assert np.array_equal(TR.dropout_keep(9, 0.5, 1, 2, start=far + 3), TR.dropout_keep(12, 0.5, 1, 2, start=far)[3:])


def test_dropped_values_are_zero_whatever_they_were():
    x = np.array([[np.inf, np.nan, -np.inf, 1.0] * 64], dtype=np.float32)
    keep = TR.dropout_keep(256, 0.5, 7, 0)
    y = TR.dropout(x, 0.5, 7, 0, "float32")
    assert (y[0][~keep] == 0).all() and not np.isfinite(y[0][keep & ~np.isfinite(x[0])]).any()
    assert (y[0][keep & np.isfinite(x[0])] == 2.0).all()


def test_forms_agree():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 64)).astype(np.float32)
    res = rng.standard_normal((4, 64)).astype(np.float32)
    ar = TR.all_reduce_dropout(x, 0.25, 5, 6, "float32", res)
    shards = TR.reduce_scatter_dropout(x, 0.25, 5, 6, "float32", np.stack([res[c, 16 * c:16 * c + 16] for c in range(4)]))
    for c in range(4):
        assert np.array_equal(shards[c], ar[c, 16 * c:16 * c + 16])
    assert np.array_equal(TR.all_gather_dropout(x.reshape(4, 64)[:, :16], 0.25, 5, 6, "float32")[2],
                          TR.dropout(x[:, :16].reshape(1, 64), 0.25, 5, 6, "float32")[0])


def test_cross_entropy_closed_forms():
    # zero weights: a uniform distribution
    t = np.array([0, 6, -100, 7])
    loss, lse, dh, dw = TR.cross_entropy(np.ones((4, 3)), np.zeros((7, 3)), t, np.ones(4))
    assert np.allclose(lse, math.log(7)) and np.allclose(loss, [math.log(7)] * 2 + [0, 0]) and not dh.any()
    want = np.full((7, 3), 2 / 7)
    want[0] -= 1
    want[6] -= 1
    assert np.allclose(dw, want)


def test_cross_entropy_gradient_against_differences():
    rng = np.random.default_rng(4)
    h, w = rng.standard_normal((3, 5)), rng.standard_normal((11, 5))
    t, g = np.array([3, 50, 10]), rng.standard_normal(3)
    _, _, dh, dw = TR.cross_entropy(h, w, t, g)
    f = lambda a, b: float((TR.cross_entropy(a, b, t)[0] * g).sum())
    eps = 1e-6
    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = eps
        assert abs((f(h + d, w) - f(h - d, w)) / (2 * eps) - dh[i]) < 1e-7
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = eps
        assert abs((f(h, w + d) - f(h, w - d)) / (2 * eps) - dw[i]) < 1e-7
