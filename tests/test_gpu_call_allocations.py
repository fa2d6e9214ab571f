"""A call on another stream while kernels on the current one still write memory
that the caller has just freed: outputs and workspaces that the binding
allocates must not be that memory."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import collective_communication_reduction_way_amd as mod

    mod.lib()
    return mod


def test_handle_of_the_null_stream(rr):
    """A handle of 0 while another stream is the current one."""
    p, T, d, V = 2, 300, 128, 2500
    h = torch.randn(T, d, device="cuda").bfloat16()
    w = [torch.randn(V // p, d, device="cuda").bfloat16() for _ in range(p)]
    t = torch.randint(0, V, (T,), device="cuda")
    loss, lse = rr.vocab_cross_entropy(h, w, t)
    assert torch.cuda.default_stream().cuda_stream == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        leave_pending_writes([T * 4, rr.vocab_cross_entropy_workspace_size(p, T, d, V, torch.bfloat16)])
        loss2, lse2 = rr.vocab_cross_entropy(h, w, t, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(loss2, loss) and torch.equal(lse2, lse)


def leave_pending_writes(sizes):
    """Blocks of these sizes, freed while their fills wait behind a bounded spin on the current stream."""
    blocks = [torch.empty(nb, dtype=torch.uint8, device="cuda") for nb in sizes for _ in range(3)]
    torch.cuda._sleep(40_000_000)
    for b in blocks:
        b.fill_(0xFF)


@pytest.mark.parametrize("as_handle", (False, True))
def test_cross_entropy_outputs_and_workspaces(rr, as_handle):
    p, T, d, V = 2, 300, 128, 2500
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    w = [torch.randn(V // p, d, generator=gen, device="cuda").bfloat16() for _ in range(p)]
    t = torch.randint(0, V, (T,), generator=gen, device="cuda")
    g = torch.rand(T, generator=gen, device="cuda")
    loss, lse = rr.vocab_cross_entropy(h, w, t)
    dh, dw = rr.vocab_cross_entropy_grad(h, w, t, lse, g)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_handle else side
    need = [rr.vocab_cross_entropy_workspace_size(p, T, d, V, torch.bfloat16, grad=k) for k in (False, True)]
    torch.cuda.synchronize()
    leave_pending_writes([T * 4, dh.numel() * 2, dw[0].numel() * 2] + need)
    loss2, lse2 = rr.vocab_cross_entropy(h, w, t, stream=stream)
    dh2, dw2 = rr.vocab_cross_entropy_grad(h, w, t, lse2, g, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(loss2, loss) and torch.equal(lse2, lse)
    assert torch.equal(dh2, dh) and all(torch.equal(a, b) for a, b in zip(dw2, dw))


@pytest.mark.parametrize("algo,group", [("ring_staged", 0), ("hier_staged", 4)])
def test_all_reduce_workspaces(rr, algo, group):
    p, n = 8, (1 << 18) + 24
    x = torch.randn(p, n, device="cuda").bfloat16()
    want, out = torch.empty_like(x), torch.empty_like(x)
    rr.all_reduce(x, want, algo=algo, group_size=group)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    leave_pending_writes([rr.workspace_size(algo, p, group, n, torch.bfloat16)])
    rr.all_reduce(x, out, algo=algo, group_size=group, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
