"""The gated projections on buffers that are off 16-byte alignment though their
rows are whole 16 bytes: other kernels, or copies in pieces, and so another order
of the sums, within the same tolerance (test_gpu_gated_linear); the same bits among
themselves, in every call and in products that are computed again."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_gated_linear import DTYPES, check_all, make, rr, run  # noqa: E402, F401


def moved(t, by):
    base = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    base[by:].copy_(t.flatten())
    return base[by:].view(t.shape)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 40, 128, 320), (2, 100, 128, 320), (3, 70, 2048, 1500), (1, 128, 1024, 4096),
                                   (2, 150, 128, 320), (2, 200, 4096, 9000), (1, 700, 2048, 9000)], ids=str)
def test_buffers_off_alignment(rr, shape, dtype):  # noqa: F811
    d = make(sum(shape), *shape, dtype)
    aligned = run(rr, d, "silu")
    check_all(aligned, d, "silu", dtype)
    first = None
    for by, names in ((1, ("x", "gate", "up", "dh")), (3, ("x",)), (2, ("gate",)), (1, ("up", "dh"))):
        e = dict(d)
        for name in names:
            e[name] = moved(d["x"], by) if name == "x" else [moved(t, by) for t in d[name]]
        got = run(rr, e, "silu")
        check_all(got, e, "silu", dtype)
        again = run(rr, e, "silu", kept=False)
        for k in got:
            assert torch.equal(got[k], again[k]), (k, names)
        first = first or got
        for k in got:
            assert torch.equal(got[k], first[k]), (k, names)
    # where dh alone lies off alignment nothing is read otherwise
    got = run(rr, dict(d, dh=[moved(t, 1) for t in d["dh"]]), "silu")
    for k in got:
        assert torch.equal(got[k], aligned[k]), k
