"""Refusals of the training operators on the CPU: every invalid argument returns
its status before any HIP call (the pointers are never dereferenced)."""

import ctypes

import pytest

import collective_communication_reduction_way_amd as rr

INVALID, UNSUPPORTED = 1, 2
FAKE = 1 << 40


def ptrs(base, p, stride=1 << 24):
    return rr._ptr_array([base + r * stride for r in range(p)])


def drop(d=0.1, dev=None):
    return rr._Dropout(d, 1, 2, dev)


FORMS = ("rr_all_reduce_dropout", "rr_reduce_scatter_dropout", "rr_dropout", "rr_all_gather_dropout")


def call(form, p=4, n=1024, dt=2, params=None, send="x", res=None, recv="y"):
    L = rr.lib()
    send = ptrs(FAKE, max(p, 1)) if send == "x" else send
    recv = ptrs(FAKE + (1 << 36), max(p, 1)) if recv == "y" else recv
    args = [send, recv, p, n, dt, params or drop(), None]
    if form != "rr_all_gather_dropout":
        args.insert(1, res)
    return getattr(L, form)(*args), L.rr_last_error().decode()


@pytest.mark.parametrize("form", FORMS)
def test_dropout_refusals(form):
    assert call(form, p=0)[0] == INVALID and call(form, p=65)[0] == INVALID
    assert call(form, dt=0)[0] == UNSUPPORTED and call(form, dt=9)[0] == UNSUPPORTED
    for d in (-0.1, 1.0, 1.5, float("nan"), float("inf")):
        st, msg = call(form, params=drop(d))
        assert st == INVALID and "drop" in msg
    st, msg = call(form, params=drop(0.1, FAKE + 4))
    assert st == INVALID and "offset_dev" in msg
    assert call(form, send=None)[0] == INVALID and call(form, recv=None)[0] == INVALID
    assert call(form, send=rr._ptr_array([FAKE, 0, FAKE, FAKE]))[0] == INVALID
    st, msg = call(form, send=ptrs(FAKE + 1, 4))
    assert st == INVALID and "aligned" in msg
    assert call(form, n=(1 << 56) + 4)[0] == INVALID
    # outputs that overlap each other, or another rank's input
    assert call(form, recv=ptrs(FAKE + (1 << 36), 4, 16))[0] == INVALID
    assert call(form, recv=ptrs(FAKE + (1 << 24), 4))[0] == INVALID
    assert call(form, n=0)[0] == 0


@pytest.mark.parametrize("form", ("rr_reduce_scatter_dropout", "rr_all_gather_dropout"))
def test_sharded_forms_need_equal_shards(form):
    st, msg = call(form, n=1022)
    assert st == INVALID and "divisible" in msg


@pytest.mark.parametrize("form", FORMS[:3])
def test_residual_refusals(form):
    assert call(form, res=rr._ptr_array([FAKE, 0, FAKE, FAKE]))[0] == INVALID
    out = FAKE + (1 << 36)
    # rank 1's residual lies over rank 0's output
    assert call(form, res=rr._ptr_array([FAKE, out, FAKE, FAKE]))[0] == INVALID
    # one residual for all ranks that is also an output
    assert call(form, res=rr._ptr_array([out] * 4))[0] == INVALID
    # shifted against its own output
    assert call(form, res=rr._ptr_array([out + 16, FAKE, FAKE, FAKE]))[0] == INVALID


def ce(grad=False, p=4, T=100, d=64, V=1000, dt=2, tb=8, hidden=FAKE, weights="w", targets=FAKE + (1 << 30),
       loss=FAKE + (1 << 31), lse=FAKE + (1 << 32), dh=FAKE + (1 << 33), dw="dw", ws=FAKE + (1 << 38), wsb=1 << 40):
    L = rr.lib()
    weights = ptrs(FAKE + (1 << 34), max(p, 1)) if weights == "w" else weights
    dw = ptrs(FAKE + (1 << 35), max(p, 1)) if dw == "dw" else dw
    if grad:
        st = L.rr_vocab_cross_entropy_grad(hidden, weights, targets, tb, lse, loss, dh, dw, p, T, d, V, dt, ws, wsb, None)
    else:
        st = L.rr_vocab_cross_entropy(hidden, weights, targets, tb, loss, lse, p, T, d, V, dt, ws, wsb, None)
    return st, L.rr_last_error().decode()


@pytest.mark.parametrize("grad", (False, True))
def test_cross_entropy_refusals(grad):
    assert ce(grad, p=0)[0] == INVALID and ce(grad, p=65)[0] == INVALID
    assert ce(grad, dt=0)[0] == UNSUPPORTED and ce(grad, dt=4)[0] == UNSUPPORTED
    for kw in (dict(d=0), dict(V=0), dict(d=(1 << 20) + 1), dict(V=(1 << 23) + 1), dict(T=(1 << 23) + 1),
               dict(d=1 << 20, V=1 << 17), dict(d=1 << 20, T=1 << 17)):
        assert ce(grad, **kw)[0] == INVALID, kw
    assert ce(grad, tb=2)[0] == INVALID and ce(grad, tb=0)[0] == INVALID
    assert ce(grad, hidden=None)[0] == INVALID and ce(grad, targets=None)[0] == INVALID
    assert ce(grad, weights=None)[0] == INVALID
    assert ce(grad, weights=rr._ptr_array([FAKE + (1 << 34), 0, 0, 0]))[0] == INVALID
    assert ce(grad, loss=None)[0] == INVALID and ce(grad, lse=None)[0] == INVALID
    assert ce(grad, hidden=FAKE + 1)[0] == INVALID and ce(grad, targets=FAKE + (1 << 30) + 4)[0] == INVALID
    assert ce(grad, loss=FAKE + (1 << 31) + 2)[0] == INVALID
    assert ce(grad, ws=None)[0] == INVALID and ce(grad, ws=FAKE + (1 << 38) + 8)[0] == INVALID
    need = rr.lib().rr_vocab_cross_entropy_workspace_size(4, 100, 64, 1000, 2, int(grad))
    st, msg = ce(grad, wsb=need - 1)
    assert st == INVALID and "workspace" in msg
    # a workspace over an input, an output over an input
    assert ce(grad, ws=FAKE - (1 << 10))[0] == INVALID
    if grad:
        assert ce(grad, dh=FAKE)[0] == INVALID
        assert ce(grad, dh=None, dw=None)[0] == INVALID
        assert ce(grad, dw=ptrs(FAKE + (1 << 34), 4))[0] == INVALID
        assert ce(grad, dw=rr._ptr_array([FAKE + (1 << 35)] * 4))[0] == INVALID
    else:
        assert ce(grad, loss=FAKE)[0] == INVALID
        assert ce(grad, loss=FAKE + (1 << 32) + 8)[0] == INVALID
        assert ce(grad, T=0, hidden=None, targets=None, loss=None, lse=None)[0] == 0


def test_workspace_size():
    L = rr.lib()
    f = L.rr_vocab_cross_entropy_workspace_size
    assert f(4, 100, 0, 1000, 2, 0) == 0 and f(0, 100, 64, 1000, 2, 0) == 0 and f(4, 100, 64, 1000, 0, 1) == 0
    assert f(4, 100, 64, 1000, 2, 0) > 0 and f(4, 100, 64, 1000, 2, 1) > 0
    # the gradient keeps one part of the logits' gradient: far below [tokens, vocab]
    assert f(8, 1 << 16, 1024, 1 << 18, 2, 1) < (1 << 16) * (1 << 18) * 2 // 16
    assert rr.vocab_cross_entropy_workspace_size(8, 2048, 4096, 50257, "bfloat16") == f(8, 2048, 4096, 50257, 2, 0)


def test_binding_refusals():
    import torch

    h, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for w in ([torch.zeros(5, 7)], [torch.zeros(3, 8), torch.zeros(1, 8)], [], [torch.zeros(5, 8).t()],
              [torch.zeros(5, 8, dtype=torch.bfloat16)]):
        with pytest.raises(ValueError):
            rr.vocab_cross_entropy(h, w, t)
    with pytest.raises(TypeError):
        rr.vocab_cross_entropy(h, [torch.zeros(5, 8)], t.short())
    with pytest.raises(ValueError):
        rr.vocab_cross_entropy(h, [torch.zeros(5, 8)], t[:3])
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        rr.all_reduce_dropout(x, torch.zeros(2, 9))
    with pytest.raises(ValueError):
        rr.all_reduce_dropout(x, torch.zeros(2, 8), residuals=[torch.zeros(8)])
    with pytest.raises(ValueError):
        rr.all_reduce_dropout(x, torch.zeros(2, 8), offset_dev=torch.zeros(1))
    with pytest.raises(ValueError):
        rr.reduce_scatter_dropout(x, torch.zeros(2, 5))
    with pytest.raises(ValueError):
        rr.all_gather_dropout(x, torch.zeros(2, 15))
