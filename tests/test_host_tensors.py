"""Host tensors are refused, with a stream given as well, by the calls that need a
workspace of the binding's and by those of the training step (no GPU needed): a
kernel that reads or writes pageable memory would fault."""

import pytest

import collective_communication_reduction_way_amd as rr

torch = pytest.importorskip("torch")


def calls():
    x, y = torch.zeros(4, 8), torch.zeros(4, 8)
    s = torch.zeros(4, 2)
    h, w, t = torch.zeros(3, 8), [torch.zeros(5, 8)], torch.zeros(3, dtype=torch.int64)
    v = torch.zeros(3)
    return {
        "all_reduce_staged": lambda k: rr.all_reduce(x.bfloat16(), y.bfloat16(), algo="ring_staged", stream=k),
        "all_reduce_hier": lambda k: rr.all_reduce_hier(x, y, group_size=2, staged=True, stream=k),
        "all_reduce_dropout": lambda k: rr.all_reduce_dropout(x, y, stream=k),
        "reduce_scatter_dropout": lambda k: rr.reduce_scatter_dropout(x, s, stream=k),
        "dropout": lambda k: rr.dropout(x, y, stream=k),
        "all_gather_dropout": lambda k: rr.all_gather_dropout(s, y, stream=k),
        "vocab_cross_entropy": lambda k: rr.vocab_cross_entropy(h, w, t, stream=k),
        "vocab_cross_entropy_grad": lambda k: rr.vocab_cross_entropy_grad(h, w, t, v, v, stream=k),
    }


@pytest.mark.parametrize("stream", (None, 4096))
@pytest.mark.parametrize("name", sorted(calls()))
def test_host_tensors_are_refused(name, stream):
    with pytest.raises(ValueError, match="GPU tensors"):
        calls()[name](stream)
