"""The norm of rows near the ends of its range: as good as that of any other row
(tolerances: test_gpu_layer_norm)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_layer_norm import DTYPES, bounds, check, check_all, make, reference, rr, run  # noqa: E402, F401

DIMS = (7, 64, 515, 768, 1024, 1027, 2048, 4096, 4104, 9001, 16384)
# sizes of a row's values, of which some are 10 times as large: with an eps 32 squares have to fit
# float32, values below 3e18; without one the sum of all, values below 1e17 at 16384 of them
LARGE = (-40, -12, 0, 30, 50, 55, 56, 57, 58)
PLAIN = (-56, -50, -40, -30, 0, 30, 50, 53)


@pytest.mark.parametrize("dtype", ("float32", "bfloat16"))
@pytest.mark.parametrize("center", (True, False))
@pytest.mark.parametrize("sizes,eps", [(LARGE, 1e-5), (LARGE, 1e-20), (PLAIN, 0.0)], ids=["usual", "small", "none"])
@pytest.mark.parametrize("dim", DIMS)
def test_rows_of_any_size(rr, dim, sizes, eps, center, dtype):  # noqa: F811
    d = make(dim, 2, len(sizes), dim, dtype)
    size = torch.tensor([2.0 ** s for s in sizes], dtype=torch.float64, device="cuda")[:, None]
    for x in d["x"]:
        x.copy_((x.double() * size).to(x.dtype))  # exact
    check_all(run(rr, d, center, eps), d, center, eps, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", (64, 4096, 16384))
def test_large_rows_beside_eps(rr, dim, dtype):  # noqa: F811
    """Values of about 5e17, in float16 of 2e4, with the usual eps; float16's smallest ones without."""
    d = make(dim, 1, 5, dim, dtype)
    for i, center in enumerate((True, False)):
        big = dict(d, x=[(t.double() * (2.0 ** 12 if dtype == "float16" else 2.0 ** 58)).to(t.dtype) for t in d["x"]])
        check_all(run(rr, big, center, 1e-5), big, center, 1e-5, dtype)
    if dtype == "float16":
        small = dict(d, x=[(t.double() * 2.0 ** -20).to(t.dtype) for t in d["x"]])
        got, e = run(rr, small, False, 0.0), reference(small, False, 0.0)
        lim, top = bounds(e, dtype, 5), torch.finfo(DTYPES[dtype]).max
        for name in ("y", "dw", "db"):
            check(name, got[name], e[name], lim[name])
        # rstd is about 2^19, dx beyond 65504 in most entries and rightly infinite there
        check("dx", got["dx"].clamp(-top, top), e["dx"].clamp(-top, top), lim["dx"])


def test_rows_between_others(rr):  # noqa: F811
    """Large rows beside ordinary ones, which keep their bits."""
    d = make(4, 1, 3000, 1024, "bfloat16")
    want = run(rr, d, True, 1e-5)
    d["x"][0][::7] *= 2.0 ** 58
    got = run(rr, d, True, 1e-5)
    check_all(got, d, True, 1e-5, "bfloat16")
    keep = torch.arange(3000, device="cuda") % 7 != 0
    assert torch.equal(got["y"][0][keep], want["y"][0][keep]) and torch.equal(got["dx"][0][keep], want["dx"][0][keep])
