"""Where the binding allocates what a call writes (no GPU: torch's streams are
stood in for).  Workspaces and outputs of a call on a given stream must come
from that stream's pool: a block from the current stream's pool may still be
written by kernels queued there, which nothing orders before the call's."""

import contextlib
from types import SimpleNamespace

import pytest

import collective_communication_reduction_way_amd as rr

torch = pytest.importorskip("torch")


class FakeTensor:
    def __init__(self, pool, shape, dtype):
        self.pool, self.shape, self.dtype, self.used_by = pool, shape, dtype, []

    def record_stream(self, stream):
        self.used_by.append(stream)


@pytest.fixture
def streams(monkeypatch):
    """torch.empty says on which stream it allocated; integer handles become their stream's name."""
    state = {"current": "current"}

    @contextlib.contextmanager
    def on(stream):
        before, state["current"] = state["current"], stream
        yield
        state["current"] = before

    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: FakeTensor(state["current"], shape, dtype))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state["current"])
    # (a handle of 0 makes torch take some stream of its own instead of the null stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda handle, device=None: f"stream {handle}" if handle else "any stream")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "null stream")
    return state


@pytest.mark.parametrize("stream,pool", [(None, "current"), ("side", "side"), (77, "stream 77"), (0, "null stream")])
def test_allocations_come_from_the_calls_stream(streams, stream, pool):
    t = SimpleNamespace(device=torch.device("cuda", 0))
    ws = rr._call_workspace(1 << 20, t, stream)
    assert ws.pool == pool and ws.shape == 1 << 20 and ws.dtype is torch.uint8
    out = rr._call_output(t, (5, 3), torch.float32, stream)
    assert out.pool == pool and out.shape == (5, 3) and out.dtype is torch.float32
    # the caller reads the output on the current stream: its block waits for those reads when it is freed
    assert out.used_by == ([] if stream is None else ["current"])
    assert streams["current"] == "current"
