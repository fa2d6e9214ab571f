"""The cross entropy at the ends of its documented sizes: the longest rows, the
widest vocabulary, many tokens; elementwise against float64 on the GPU."""

import pytest

from test_gpu_vocab_pieces import DT, bounds, check, inputs, rr  # noqa: F401 (rr: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ("float32", "bfloat16", "float16"))
@pytest.mark.parametrize("p,T,d,V", [
    (2, 3, 1 << 20, 70),
    (1, 2, (1 << 20) - 1, 40),
    (3, 2, 8, 1 << 23),
    (64, 1, 7, (1 << 20) + 63),
    (2, (1 << 20) + 1, 8, 70),
    (3, 300000, 9, 65),
])
def test_ends_of_the_sizes(rr, p, T, d, V, dtype):
    h, w, t, g = inputs(p, T, d, V, dtype, 1, 0)
    loss, lse = rr.vocab_cross_entropy(h, w, t)
    dh, dw = rr.vocab_cross_entropy_grad(h, w, t, lse, g)
    want, tol = bounds(h, w, t, g, dtype, V + 4)
    check(loss, want[0], tol[0], "loss")
    check(lse, want[1], tol[1], "lse")
    check(dh, want[2], tol[2], "dhidden")
    check(torch.cat(dw), want[3], tol[3], "dweights")
    del want, tol, h, w, dh, dw
    torch.cuda.empty_cache()


def test_past_the_ends_is_refused(rr):
    one = torch.zeros(1, dtype=torch.int64, device="cuda")
    with pytest.raises(rr.RRError):
        rr.vocab_cross_entropy(torch.zeros(1, (1 << 20) + 1, device="cuda"), [torch.zeros(4, (1 << 20) + 1, device="cuda")],
                               one, workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))
    with pytest.raises(rr.RRError):
        rr.vocab_cross_entropy(torch.zeros(1, 1, device="cuda"), [torch.zeros((1 << 23) + 1, 1, device="cuda")], one,
                               workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))
