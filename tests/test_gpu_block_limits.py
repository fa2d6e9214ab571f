"""The norm and the gated projections at the ends of their sizes, with buffers
given twice, and from two threads at once (tolerances: test_gpu_gated_linear,
test_gpu_layer_norm)."""

import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_gated_linear import DTYPES, check_all, make, rr, run  # noqa: E402, F401


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 300, 2 ** 20, 70), (1, 3, 2 ** 20, 40), (1, 90, 2 ** 20 - 1, 9), (2, 130, 64, 2 ** 19),
                                   (1, 2, 64, 2 ** 19), (64, 66, 24, 2 ** 19 - 5)], ids=str)
def test_widest_rows_and_most_features(rr, shape, dtype):  # noqa: F811
    d = make(sum(shape) % 1000, *shape, dtype)
    want = run(rr, d, "silu")
    check_all(want, d, "silu", dtype)
    again = run(rr, d, "silu", kept=False)
    for k in want:
        assert torch.equal(again[k], want[k]), k


def test_most_rows(rr):  # noqa: F811
    """2^31 - 1 rows of one value: x / sqrt(x^2 + eps), and the gradient that joins a residual."""
    rows, eps, part = 2 ** 31 - 1, 0.25, 1 << 27
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x, dy = (torch.empty(1, rows, 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (x, dy):
        for lo in range(0, rows, part):
            v = t[0, lo:lo + part]
            v.copy_(torch.randn(v.shape, generator=gen, device="cuda"))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(rows, device="cuda")
    rr.layer_norm(x, None, None, y, eps=eps, center=False, rstd=rstd)
    _, dw, db = rr.layer_norm_grad(dy, x, None, None, rstd, dx, residuals=dy, center=False)
    h, u = 2.0 ** -8, 2.0 ** -24
    sums = torch.zeros(4, dtype=torch.float64, device="cuda")
    for lo in range(0, rows, part):
        xs, gs = x[0, lo:lo + part].double(), dy[0, lo:lo + part].double()
        r = (xs.square() + eps).rsqrt()
        xh = xs * r
        assert ((rstd[lo:lo + part].double() - r[:, 0]).abs() <= 4 * u * r[:, 0]).all()
        assert ((y[0, lo:lo + part].double() - xh).abs() <= (h + 8 * u) * xh.abs() + 2.0 ** -133).all()
        # dx = r (g - xh (g xh)) + g, four roundings each of terms of size r |g| and below
        want = r * (gs - xh * (gs * xh)) + gs
        assert ((dx[0, lo:lo + part].double() - want).abs() <= h * want.abs() + 32 * u * (1 + r) * gs.abs() + 2.0 ** -133).all()
        sums += torch.stack([(gs * xh).sum(), gs.sum(), (gs * xh).abs().sum(), gs.abs().sum()])
    # a thread adds 2^31 / 4096 terms in turn, then 8 groups and 512 parts
    lim = (2 ** 19 + 64) * u
    assert abs(dw.double() - sums[0]) <= lim * sums[2] + h * sums[0].abs()
    assert abs(db.double() - sums[1]) <= lim * sums[3] + h * sums[1].abs()


def test_buffers_given_twice(rr):  # noqa: F811
    """One matrix as gate and up of every rank, one gradient of every rank's output, one residual."""
    d = make(5, 3, 170, 136, 210, "bfloat16")
    d["gate"] = d["up"] = [d["gate"][0]] * 3
    d["dh"] = [d["dh"][0]] * 3
    want = run(rr, d, "gelu")
    check_all(want, d, "gelu", "bfloat16")
    one = want["dg"].view(3, 70, 136)
    assert torch.equal(one[0], one[1]) and torch.equal(one[0], one[2])
    x = [d["x"], d["x"]]
    y = [torch.empty_like(d["x"]) for _ in range(2)]
    mean, rstd = (torch.empty(2, 170, device="cuda") for _ in range(2))
    rr.layer_norm(x, None, None, y, mean=mean, rstd=rstd)
    assert torch.equal(y[0], y[1]) and torch.equal(mean[0], mean[1])
    dx, dw, db = rr.layer_norm_grad(x, x, None, mean, rstd, residuals=x)
    assert torch.equal(dx[0], dx[1]) and torch.isfinite(dw.float()).all()


def test_two_threads(rr):  # noqa: F811
    """Calls of two threads, each on a stream of its own: the same bits as alone."""
    cases = [(make(9, 2, 300, 264, 500, "bfloat16"), "silu"), (make(10, 3, 90, 770, 410, "float16"), "gelu")]
    want = [run(rr, d, act) for d, act in cases]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            d, act = cases[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i].append(run(rr, d, act))
                    x = d["x"].clone()
                    rr.layer_norm([x], None, None)
                    with pytest.raises(ValueError):
                        rr.layer_norm([x], None, None, [x, x])
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        assert len(got[i]) == 20
        for one in got[i]:
            for k in want[i]:
                assert torch.equal(one[k], want[i][k]), (i, k)
