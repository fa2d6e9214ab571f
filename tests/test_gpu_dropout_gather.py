"""The gather with dropout above 128 MiB written, where several workgroups read
a shard's block: shards that end inside a group of 16 bytes, rank buffers off
16-byte alignment, every type, bit for bit against the oracle; outputs between
sentinels, inputs between NaN."""

import numpy as np
import pytest

import workloads as W
from gpu_util import assert_bitwise, to_dev, to_host
from oracle import training as TR
from test_gpu_guard import Guarded
from test_gpu_training_guard import among_nan, rr  # noqa: F401 (rr: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SEED, OFFSET = 0xFEDCBA9876543210, (3 << 34) + 1


@pytest.mark.parametrize("dtype,p,m,shift", [
    ("bfloat16", 8, (1 << 20) + 41, 0),
    ("bfloat16", 7, 1400003, 1),
    ("bfloat16", 9, 900007, 5),
    ("float16", 8, (1 << 20) + 43, 0),
    ("float16", 3, 7500001, 3),
    ("float32", 8, (1 << 19) + 21, 0),
    ("float32", 7, 700001, 1),
    ("float32", 2, 8400006, 2),
    ("float32", 64, 8195, 3),
])
def test_ragged_shards(rr, dtype, p, m, shift):
    n, esz = p * m, 4 if dtype == "float32" else 2
    assert p * n * esz > 128 << 20
    x = W.random_inputs(61, p, m, dtype)
    xs = [among_nan(to_dev(r, dtype), shift) for r in x]
    want = TR.all_gather_dropout(x, 0.35, SEED, OFFSET, dtype)
    g = Guarded([n * esz] * p, dtype, shift * esz)
    rr.all_gather_dropout(xs, g.views(), drop=0.35, seed=SEED, offset=OFFSET)
    torch.cuda.synchronize()
    what = f"{dtype} p={p} m={m} shift={shift}"
    g.check_guards(what)
    for r in range(p):
        assert_bitwise(to_host(g.view(r), dtype), want[r], what)
    # in place, where one workgroup writes every destination
    full = [v.view(n) for v in g.views()]
    for r, (v, s) in enumerate(zip(full, xs)):
        v.fill_(float("nan"))
        v[r * m:(r + 1) * m].copy_(s)
    rr.all_gather_dropout([v[r * m:(r + 1) * m] for r, v in enumerate(full)], full, drop=0.35, seed=SEED, offset=OFFSET)
    torch.cuda.synchronize()
    g.check_guards(what)
    for r in range(p):
        assert_bitwise(to_host(g.view(r), dtype), want[r], what + " in place")
