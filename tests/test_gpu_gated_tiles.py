"""The gated projections in shapes that take the largest tiles in every use: with
products kept in either type or computed again, dhidden whole, in parts and in pieces, the
weights' gradients with and without small tiles behind the large ones (test_gated_plan
says which shape takes what; tolerances: test_gpu_gated_linear)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gated_plan import SHAPES, plan  # noqa: E402
from test_gpu_gated_linear import DTYPES, check_all, make, rr, run  # noqa: E402, F401


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_large_tiles_in_every_use(rr, shape, dtype):  # noqa: F811
    assert plan(*shape, dtype) == SHAPES[shape][dtype != "float32"]
    act = ("silu", "gelu")[sum(shape) % 2]
    d = make(sum(shape), *shape, dtype)
    want = run(rr, d, act)
    check_all(want, d, act, dtype)
    again = run(rr, d, act, kept=False)
    for k in want:
        assert torch.equal(again[k], want[k]), k
    del again
    h = torch.cat(rr.gated_linear(d["x"], d["gate"], d["up"], activation=act), 1)
    assert torch.equal(h, want["h"])
    if dtype != "float32":
        check_all(run(rr, d, act, pre=DTYPES[dtype]), d, act, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 2060, 280, 16635), (2, 1289, 1345, 18386), (1, 763, 393, 17384)], ids=str)
def test_nothing_outside_is_written(rr, shape, dtype):  # noqa: F811
    """Outputs and workspace between sentinels, the workspace full of NaN."""
    p, tokens, dim, ffn = shape
    dt, pad = DTYPES[dtype], 64
    d = make(3, *shape, dtype)
    want = run(rr, d, "silu")
    guards = []

    def guarded(rows, cols, kind=dt):
        base = torch.full((rows * cols + 2 * pad,), 77.0, dtype=kind, device="cuda")
        guards.append(base)
        return base[pad:pad + rows * cols].view(rows, cols)

    n = [w.shape[0] for w in d["gate"]]
    h = [guarded(tokens, k) for k in n]
    a, u = ([guarded(tokens, k, torch.float32) for k in n] for _ in range(2))
    dg, du = ([guarded(k, dim) for k in n] for _ in range(2))
    dx = guarded(tokens, dim)
    for kept in (True, False):
        spaces = []
        for grad in (False, True):
            need = rr.gated_linear_workspace_size(p, tokens, dim, ffn, dt, grad=grad, kept=kept)
            spaces.append((torch.full((need + 2 * pad,), 0xFF, dtype=torch.uint8, device="cuda"), need))
        rr.gated_linear(d["x"], d["gate"], d["up"], h, pre_gates=a, pre_ups=u,
                        workspace=spaces[0][0][pad:pad + spaces[0][1]])
        pre = dict(pre_gates=a, pre_ups=u) if kept else {}
        rr.gated_linear_grad(d["x"], d["gate"], d["up"], d["dh"], dhidden=dx, dgate_weights=dg, dup_weights=du,
                             workspace=spaces[1][0][pad:pad + spaces[1][1]], **pre)
        got = {"h": torch.cat(h, 1), "a": torch.cat(a, 1), "u": torch.cat(u, 1), "dx": dx, "dg": torch.cat(dg),
               "du": torch.cat(du)}
        for k in want:
            assert torch.equal(got[k], want[k]), (k, kept)
        for base, need in spaces:
            assert (base[:pad] == 0xFF).all() and (base[pad + need:] == 0xFF).all()
        for base in guards:
            assert (base[:pad] == 77).all() and (base[-pad:] == 77).all()
            base[pad:-pad] = 3.0
