"""float16 gradients of the output weight where the tokens' loss gradients and
hidden states are of very different sizes, against the definition in float64.

Tolerances.  u = 2^-11 (half a float16 step), f = 2^-23 (a unit of a float32
sum).  The hidden row of token t is kept as float16 times 2^(e_t - m + 15), with
|g_t| < 2^e_t, |h_t| < 2^a_t and m the largest e_t + a_t.  That is a power of
two, so only values below 2^-14 are rounded, to a multiple of 2^-24: off by at
most 2^-25, which is g_t h_t off by 2^(m - 40).  The gradient of a logit is kept
as float16 times 2^(15 - e_t): off by u of itself (the target's entry by u^2) and,
below 2^-14, by 2^-25 (2^-39 of |g|, which is 2^(e_t - 1) at least) or by itself
where that is less.  The sums of the products
are off by (T + 4) f of their magnitudes, the result by u of itself and 2^-25.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U, F = 2.0 ** -11, 2.0 ** -23


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import collective_communication_reduction_way_amd as mod

    mod.lib()
    return mod


def exponent(x):
    """The smallest e with |x| < 2^e."""
    return np.frexp(np.abs(x))[1]


def definition(h, w, t, g):
    """Float64 gradients of all tokens' losses and the tolerance of dweights."""
    T, d = h.shape
    z = h @ w.T
    lse = np.log(np.exp(z - z.max(axis=1, keepdims=True)).sum(axis=1)) + z.max(axis=1)
    P = np.exp(z - lse[:, None])
    hot = np.zeros_like(P)
    hot[np.arange(T), t] = 1
    ga = np.abs(g)[:, None]
    G = P - hot
    # logits and statistics in float32, as a relative error of the probabilities
    Z = ((d + 2) * F * (np.abs(h) @ np.abs(w).T)).max(axis=1)
    L = Z + 16 * F * (np.log(w.shape[0]) + np.abs(lse) + 4)
    kept = np.where(hot > 0, U * U, U) * np.abs(G) + np.minimum(np.abs(G), 2.0 ** -39)
    dG = ga * (P * (Z + L + 6 * F)[:, None] + kept)
    m = (exponent(g) + exponent(np.abs(h).max(axis=1))).max()
    dw = (G * g[:, None]).T @ h
    tol = (dG.T @ np.abs(h) + (np.abs(G).sum(axis=0) * 2.0 ** (m - 40))[:, None]
           + (T + 4) * F * ((np.abs(G) * ga).T @ np.abs(h)) + U * np.abs(dw) + 2.0 ** -25)
    return dw, tol


def two_kinds(T, d, V, small, seed):
    """Half of the tokens and of the vocabulary are of one kind, half of the
    other, and a token gives the other kind's rows probabilities under e^-50: the
    rows of either kind get their gradient from their own tokens alone.  The
    second kind's loss gradients are `small` of the first's, and all hidden
    values but the kind's are small."""
    rng = np.random.default_rng(seed)
    h = rng.standard_normal((T, d)) * 0.02
    w = rng.standard_normal((V, d)) * 0.5
    kind_t, kind_v = np.arange(T) % 2, np.arange(V) % 2
    h[:, 0], h[:, 1] = np.where(kind_t == 0, 4.0, -4.0), 0.0
    w[:, 0], w[:, 1] = np.where(kind_v == 0, 8.0, -8.0), 0.0
    g = np.where(kind_t == 0, 2.0 ** 12, 2.0 ** 12 * small) * rng.uniform(0.6, 1.4, size=T)
    t = rng.permutation(V // 2)[:T] * 2 + kind_t
    half = lambda x: torch.from_numpy(x).half()
    return half(h), half(w), torch.from_numpy(t), torch.from_numpy(g).float()


@pytest.mark.parametrize("T,d,V,p", [(60, 72, 600, 2), (61, 70, 601, 3), (1100, 64, 3000, 2), (40, 1032, 8001, 1)])
@pytest.mark.parametrize("small", (2.0 ** -8, 2.0 ** -14, 2.0 ** -20))
def test_small_loss_gradients_of_small_hidden_states(rr, T, d, V, p, small):
    h, w, t, g = two_kinds(T, d, V, small, seed=T)
    b = [r * V // p for r in range(p + 1)]
    ws = [w[b[r]:b[r + 1]].contiguous().cuda() for r in range(p)]
    _, lse = rr.vocab_cross_entropy(h.cuda(), ws, t.cuda())
    _, dw = rr.vocab_cross_entropy_grad(h.cuda(), ws, t.cuda(), lse, g.cuda())
    want, tol = definition(h.double().numpy(), w.double().numpy(), t.numpy(), g.double().numpy())
    got = torch.cat(dw).double().cpu().numpy()
    assert np.isfinite(got).all()
    over = np.abs(got - want) - tol
    i = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, f"{(over > 0).sum()} of {over.size} off, worst at {i}: got {got[i]} want {want[i]} tol {tol[i]}"
    # the tolerance itself: the targets' rows of the second kind are known to three digits
    rows = t.numpy()[t.numpy() % 2 == 1]
    assert np.median(tol[rows, 2:] / np.abs(want[rows, 2:])) < (2.0 ** -9 if small >= 2.0 ** -14 else 2.0 ** -7)


def test_rows_without_a_size(rr):
    """Tokens whose hidden states or loss gradients are zero, and one whose are
    the largest numbers, beside ordinary ones."""
    T, d, V = 90, 64, 500
    h, w, t, g = two_kinds(T, d, V, 2.0 ** -4, seed=3)
    h[3], h[4] = 0, 0
    g[3], g[5], g[6] = 2.0 ** 60, 0.0, -0.0
    h[7] = 0
    h[7, 2], g[7] = 2.0 ** -24, 2.0 ** 15
    _, lse = rr.vocab_cross_entropy(h.cuda(), [w.cuda()], t.cuda())
    dh, (dw,) = rr.vocab_cross_entropy_grad(h.cuda(), [w.cuda()], t.cuda(), lse, g.cuda())
    live = np.array([i for i in range(T) if i not in (3, 5, 6)])
    want, tol = definition(h.double().numpy()[live], w.double().numpy(), t.numpy()[live], g.double().numpy()[live])
    got = dw.double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
    assert (dh[5] == 0).all() and (dh[6] == 0).all()


@pytest.mark.parametrize("T", (90, 1100))
def test_captured_steps_follow_their_inputs(rr, T):
    """The rows' scales are found again at every replay, as the sizes of hidden
    states and loss gradients change."""
    h, w, t, g = (x.cuda() for x in two_kinds(T, 72, 2400, 2.0 ** -6, seed=9))
    _, lse = rr.vocab_cross_entropy(h, [w], t)
    rr.vocab_cross_entropy_grad(h, [w], t, lse, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse2 = rr.vocab_cross_entropy(h, [w], t)
        dh2, (dw2,) = rr.vocab_cross_entropy_grad(h, [w], t, lse2, g)
    for k in range(4):
        g.mul_((1.0, 2.0 ** -9, 2.0 ** 12, -1.0)[k])
        h[:, 2:].mul_((1.0, 8.0, 0.25, 1.0)[k])
        graph.replay()
        torch.cuda.synchronize()
        _, lse = rr.vocab_cross_entropy(h, [w], t)
        dh, (dw,) = rr.vocab_cross_entropy_grad(h, [w], t, lse, g)
        assert torch.equal(lse2, lse) and torch.equal(dh2, dh) and torch.equal(dw2, dw), k
        # (|g h| reaches 1.4 * 2^15 * 4, past the largest float16: the targets' rows may be infinite)
        assert not torch.isnan(dw).any() and float(dw.abs().max()) > 0
