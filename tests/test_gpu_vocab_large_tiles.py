"""float16 through the largest tile of every product, against the definition in
float64, with the plan that the library logs; and the same sizes with targets
that are as uneven as text's, so that more of them than a tile holds at a time
share its columns."""

import re

import numpy as np
import pytest

from test_gpu_vocab import bounds, check, inputs, rr  # noqa: F401 (rr: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LARGE = "tiles=0/0/0"


def run(rr, tuning, capfd, h, w, t, g):
    loss, lse = rr.vocab_cross_entropy(h, w, t)
    tuning.set("RR_LOG", 1)
    capfd.readouterr()
    dh, dw = rr.vocab_cross_entropy_grad(h, w, t, lse, g)
    log = capfd.readouterr().err
    tuning.set("RR_LOG", 0)
    return loss, lse, dh, dw, re.search(r"tiles=\d/\d/\d", log).group(0)


def test_float16(rr, tuning, capfd):
    h, w, t, g = inputs(5, 3, 2100, 2064, 8300, "float16")
    *got, tiles = run(rr, tuning, capfd, h, w, t, g)
    assert tiles == LARGE
    want, tol = bounds(h, w, t, g, "float16")
    check(got[0], want[0], tol[0], "loss")
    check(got[1], want[1], tol[1], "lse")
    check(got[2], want[2], tol[2], "dhidden")
    check(torch.cat(got[3]), want[3], tol[3], "dweights")


@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
def test_uneven_targets(rr, tuning, capfd, dtype):
    """Row v is the target of a share of about 1 / (v + 1) of the tokens: the first
    tile has over a thousand targets, the last ones none."""
    h, w, t, g = inputs(6, 2, 2100, 2064, 8300, dtype, masked=0.0)
    share = 1.0 / (np.arange(8300) + 1.0)
    t = torch.from_numpy(np.random.default_rng(1).choice(8300, size=2100, p=share / share.sum())).cuda()
    t[::17] = -1
    assert int(((t >= 0) & (t < 256)).sum()) > 1000
    *got, tiles = run(rr, tuning, capfd, h, w, t, g)
    assert tiles == LARGE
    want, tol = bounds(h, w, t, g, dtype)
    check(got[0], want[0], tol[0], "loss")
    check(got[2], want[2], tol[2], "dhidden")
    check(torch.cat(got[3]), want[3], tol[3], "dweights")
