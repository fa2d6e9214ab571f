"""The vocabulary cross entropy where the vocabulary is walked in several pieces:
losses, statistics and both gradients elementwise against the definition in
float64 (on the GPU: these vocabularies are wide).

Pieces come from the size of the logits' gradient (1 GiB of it), from rows that
are copied into aligned ones (64 MiB of them) and from 2^20 columns; every case
says how many it is made for, and the plan that the library logs has to say the
same.

Tolerances: those of the tests of single pieces, with u = eps/2 of the storage
type and f = 2^-23, except that dhidden's sum over V is one of `depth` additions
in a row at most: a split of a piece, the pieces, the splits.  The last column of
the weights is 1 in targets' rows and 0 elsewhere and that of the hidden states
0, so that dhidden there is the target's entry alone, kept to u^2.
"""

import re

import pytest

from oracle.collectives import chunk_bounds

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
F = 2.0 ** -23


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import collective_communication_reduction_way_amd as mod

    mod.lib()
    return mod


def inputs(p, T, d, V, dtype, pieces, shift):
    gen = torch.Generator(device="cuda").manual_seed(T + d + V)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    t = torch.randint(0, V, (T,), generator=gen, device="cuda")
    # about where pieces and shards end
    edges = [V * k // pieces + j for k in range(pieces + 1) for j in (-1, 0, 1)]
    edges += [b + j for b in chunk_bounds(V, p) for j in (-1, 0)]
    edges = [e for e in edges if 0 <= e < V][:T // 2]
    t[:len(edges)] = torch.tensor(edges, device="cuda")
    w = normal(V, d) * (1.5 / d ** 0.5)
    w[:, -1] = 0
    w[t, -1] = 1
    w = w.to(DT[dtype])
    h = normal(T, d)
    h[::2] += 2.0 * w[t[::2]].float()
    h[:, -1] = 0
    h = h.to(DT[dtype])
    dead = torch.rand(T, generator=gen, device="cuda") < 0.2
    dead[0] = False  # one token counts at least
    t[dead] = -1
    g = torch.rand(T, generator=gen, device="cuda") * 3 - 1.5

    def put(x):
        buf = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")
        buf[shift:].copy_(x.reshape(-1))
        return buf[shift:].view(x.shape)

    b = chunk_bounds(V, p)
    return put(h), [put(w[b[r]:b[r + 1]]) for r in range(p)], t, g


def exponent(x):
    return torch.frexp(x.abs())[1].double()


def bounds(h, ws, t, g, dtype, depth):
    """Float64 results and their tolerances."""
    h, w, g = h.double(), torch.cat(ws).double(), g.double()
    T, d = h.shape
    V = w.shape[0]
    u = torch.finfo(DT[dtype]).eps / 2
    live = t >= 0
    hz = torch.where(live[:, None], h, 0.0)
    wt = w.t().contiguous()
    z = h @ wt
    lse = torch.logsumexp(z, dim=1)
    rows = torch.nonzero(live)[:, 0]
    zt = torch.zeros(T, dtype=torch.float64, device="cuda")
    zt[rows] = z[rows, t[rows]]
    loss = torch.where(live, lse - zt, 0.0)
    Z = ((d + 2) * F * (h.abs() @ wt.abs())).amax(dim=1)
    L = Z + 16 * F * (torch.log(torch.tensor(float(V))).item() + lse.abs() + 4)
    tl = torch.where(live, Z + L + 2 * F * loss.abs(), 0.0)
    P = z.sub_(lse[:, None]).exp_()
    gz = torch.where(live, g, 0.0)
    ga = gz.abs()[:, None]
    dG = P * (Z + L + 6 * F)[:, None]  # logits, statistics, the exponential
    P[rows, t[rows]] -= 1
    G = P.abs()
    kept = u * G
    kept[rows, t[rows]] *= u
    # float16 keeps an entry at 2^15 times its size, with steps of 2^-24, and the hidden values at up to 2^15
    tiny, m = 0.0, 0.0
    if dtype == "float16":
        kept += torch.clamp(G, max=2.0 ** -39)
        tiny = 2.0 ** -25
        m = float(torch.exp2((exponent(gz) + exponent(hz.abs().amax(dim=1)))[live].max() - 40))
    dG = (dG + kept) * ga
    dh = (P * gz[:, None]) @ w
    dw = (P * gz[:, None]).t().contiguous() @ hz
    G *= ga
    th = dG @ w.abs() + depth * F * (G @ w.abs()) + u * dh.abs() + tiny
    tw = dG.t().contiguous() @ hz.abs() + (T + 4) * F * (G.t().contiguous() @ hz.abs()) + u * dw.abs() + tiny
    if m:
        tw += m * (P.abs() * live[:, None]).sum(dim=0)[:, None]
    return (loss, lse, dh, dw), (tl, L, th, tw)


def check(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - tol
    if over.numel() and float(over.max()) > 0:
        i = int(over.argmax())
        pick = lambda x: float(x.expand(over.shape).reshape(-1)[i])
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.numel()} off, worst at {i} of {tuple(over.shape)}: "
                             f"got {pick(got)} want {pick(want)} tol {pick(tol)}")


CASES = [
    # p, tokens, dim, vocab, type, shift, pieces forward, pieces of the gradient
    # by the gradient of the logits; a shard's end at a piece's (p = 2) and inside pieces
    (2, 1000, 16, 600000, "bfloat16", 0, 1, 2),
    (3, 1000, 16, 600000, "float16", 0, 1, 2),
    (3, 2100, 16, 140000, "float32", 0, 1, 2),
    (5, 2100, 24, 561234, "bfloat16", 0, 1, 3),
    # by the columns; riders along the first piece's and the last piece's launches
    (2, 20, 64, 2000000, "bfloat16", 0, 2, 2),
    (7, 20, 64, 1100000, "float16", 0, 2, 2),
    (2, 20, 16, 1500001, "float32", 0, 2, 2),
    # by the rows that are copied: odd lengths, and aligned lengths off alignment
    (3, 40, 2050, 50257, "bfloat16", 0, 4, 4),
    (2, 300, 2050, 50257, "float32", 0, 7, 7),
    (64, 40, 4100, 20000, "float16", 0, 3, 3),
    (5, 1000, 2050, 40000, "float16", 0, 3, 3),
    (8, 2048, 770, 131072, "bfloat16", 0, 4, 4),
    (2, 33, 64, 600000, "bfloat16", 1, 2, 2),
    (3, 1, 1026, 70001, "float32", 0, 5, 5),
]


@pytest.mark.parametrize("p,T,d,V,dtype,shift,fwd,grad", CASES)
def test_pieces(rr, tuning, capfd, p, T, d, V, dtype, shift, fwd, grad):
    h, w, t, g = inputs(p, T, d, V, dtype, max(fwd, grad), shift)
    dead = t < 0
    need = [rr.vocab_cross_entropy_workspace_size(p, T, d, V, DT[dtype], grad=k) for k in (False, True)]
    ws = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in need]
    tuning.set("RR_LOG", 1)
    capfd.readouterr()
    loss, lse = rr.vocab_cross_entropy(h, w, t, workspace=ws[0])
    log = capfd.readouterr().err
    assert int(re.search(r"pieces=(\d+)", log).group(1)) == fwd, log
    # masked rows may hold anything
    h2 = h
    if shift == 0 and T > 1:
        h2 = h.clone()
        h2[dead] = float("nan")
    dh, dw = rr.vocab_cross_entropy_grad(h2, w, t, lse, g, workspace=ws[1])
    log = capfd.readouterr().err
    assert int(re.search(r"pieces=(\d+)", log).group(1)) == grad, log
    tuning.set("RR_LOG", 0)
    splits = int(re.search(r"splits=(\d+)", log).group(1))
    columns = (V + 64 * p) // grad + 256
    want, tol = bounds(h, w, t, g, dtype, columns // splits + 64 + grad + splits + 4)
    check(loss, want[0], tol[0], "loss")
    check(lse, want[1], tol[1], "lse")
    check(dh, want[2], tol[2], "dhidden")
    check(torch.cat(dw), want[3], tol[3], "dweights")
    assert (dh[dead] == 0).all()
    # either side alone
    a = rr.vocab_cross_entropy_grad(h, w, t, lse, g, need_weights=False)
    b = rr.vocab_cross_entropy_grad(h, w, t, lse, g, need_hidden=False)
    assert torch.equal(a[0], dh) and all(torch.equal(x, y) for x, y in zip(b[1], dw))
    del want, tol, a, b
    torch.cuda.empty_cache()
