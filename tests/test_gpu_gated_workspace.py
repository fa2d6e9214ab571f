"""The gated projections' gradient in exactly the workspace that its form asks
for, between sentinels and full of NaN: the same bits as with room to spare."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_gated_linear import DTYPES, make, rr  # noqa: E402, F401


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kept", (True, False))
@pytest.mark.parametrize("off", (0, 1))
@pytest.mark.parametrize("shape", [(2, 40, 100, 130), (3, 200, 330, 515), (1, 1100, 264, 300), (2, 4200, 2048, 2300)], ids=str)
def test_workspace_of_each_form(rr, shape, off, kept, dtype):  # noqa: F811
    p, tokens, dim, ffn = shape
    if dtype == "float32" and tokens == 4200:
        ffn = 700
    d = make(7, p, tokens, dim, ffn, dtype, off=off)
    n = [(tokens, w.shape[0]) for w in d["gate"]]
    a, u = ([torch.empty(s, device="cuda") for s in n] for _ in range(2))
    rr.gated_linear(d["x"], d["gate"], d["up"], pre_gates=a, pre_ups=u)
    pre = dict(pre_gates=a, pre_ups=u) if kept else {}
    results = []
    for more in (0, 1 << 20):
        need, pad = rr.gated_linear_workspace_size(p, tokens, dim, ffn, DTYPES[dtype], grad=True, kept=kept), 64
        base = torch.full((need + more + 2 * pad,), 0xFF, dtype=torch.uint8, device="cuda")
        results.append(rr.gated_linear_grad(d["x"], d["gate"], d["up"], d["dh"], workspace=base[pad:pad + need + more], **pre))
        assert (base[:pad] == 0xFF).all() and (base[pad + need:] == 0xFF).all()
    (dx, dg, du), (dx2, dg2, du2) = results
    for one, two in zip([dx, *dg, *du], [dx2, *dg2, *du2]):
        assert torch.isfinite(one.float()).all() and torch.equal(one, two)
