"""On which stream the Python layer allocates what it uses on a caller's stream
(no GPU: torch's stream context and the entry points are stand-ins)."""
import contextlib

import pytest
import torch

from sparse_mixture_experts_04_b200 import MoeLayer, api


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def streams(monkeypatch):
    """The stack of handles that torch's current stream would be; starts on 1."""
    stack = [1]

    @contextlib.contextmanager
    def on(stream):
        stack.append(stream.cuda_stream)
        yield
        stack.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    # torch makes a stream of its own for the handle 0
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: FakeStream(h or 99))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: FakeStream(stack[-1]))
    monkeypatch.setattr(api, "_current_stream", lambda dev: stack[-1])
    monkeypatch.setattr(api, "_cuda", lambda name, t: 0)
    return stack


class Recorder:
    """A layer on the CPU whose kernel only notes on which stream it was called,
    and whose workspace notes on which it was allocated."""

    def __init__(self, monkeypatch, stack):
        self.allocated, self.ran, self.recorded = [], [], []
        prob = api.make_problem(2, 16, 4, 2, 16)
        self.layer = MoeLayer(prob, {"w13": None, "w2": None}, "cpu")
        self.layer._check_weights = lambda: None
        rec = self

        class Workspace:
            def record_stream(self, s):
                rec.recorded.append(s.cuda_stream)

        def alloc(prob, device):
            rec.allocated.append(stack[-1])
            return Workspace()

        monkeypatch.setattr(api, "alloc_few_workspace", alloc)
        self.layer._forward_few = lambda prob, x, w, y, r, stats, ws, stream: rec.ran.append(
            stack[-1] if stream is None else api._stream(stream))
        self.x = torch.zeros((2, 16), dtype=torch.bfloat16)

    def call(self, stream=None):
        self.layer.forward_few(self.x, torch.empty_like(self.x), stream=stream)


@pytest.mark.parametrize("stream", [FakeStream(7), 7])
def test_the_few_token_workspace_is_cleared_on_the_stream_that_uses_it(streams, monkeypatch, stream):
    r = Recorder(monkeypatch, streams)
    r.call(stream)
    assert r.allocated == r.ran == [7] and streams == [1]
    r.call(stream)
    assert r.allocated == [7] and r.recorded == []       # once, and the same stream again
    r.call()                                             # another stream: the allocator is told
    assert r.ran == [7, 7, 1] and r.recorded == [1]


def test_the_few_token_workspace_on_the_current_stream(streams, monkeypatch):
    r = Recorder(monkeypatch, streams)
    r.call()
    r.call()
    assert r.allocated == [1] and r.ran == [1, 1] and r.recorded == []
    r.call(9)
    r.call(9)
    r.call()
    assert r.recorded == [9]                              # once for each stream


def test_no_stream_context_without_a_stream(streams):
    with api._on_stream(None, 0):
        assert streams == [1]
    with api._on_stream(3, 0):
        assert streams == [1, 3]


def test_outputs_are_allocated_on_the_stream_that_writes_them(streams, monkeypatch):
    """forward, forward_few and quantize_rows without output tensors, on a stream."""
    made, recorded = [], []

    class Out:
        device = torch.device("cpu")

        def record_stream(self, s):
            recorded.append(s.cuda_stream)

    def empty(*args, **kwargs):
        made.append(streams[-1])
        return Out()

    r = Recorder(monkeypatch, streams)
    r.layer._forward = lambda *a: None
    monkeypatch.setattr(api, "moe_quantize_rows", lambda *a: None)
    monkeypatch.setattr(torch, "empty", empty)
    for call, n in ((lambda s: r.layer.forward_few(r.x, stream=s), 1), (lambda s: r.layer.forward(r.x, stream=s), 1),
                    (lambda s: api.quantize_rows(r.x, stream=s), 2)):
        made.clear()
        recorded.clear()
        call(5)
        assert made == [5] * n and recorded == [1] * n   # written on 5, read on the current one
        made.clear()
        recorded.clear()
        call(None)
        assert made == [1] * n and recorded == []


def test_the_default_streams_handle_means_the_default_stream(streams, monkeypatch):
    r = Recorder(monkeypatch, streams)
    r.call(0)                                             # from a current stream of its own (1)
    assert r.allocated == r.ran == [0]
    with api._on_stream(FakeStream(0), 0):
        assert streams == [1, 0]


def test_backward_and_balance_update_clear_their_buffers_on_their_stream(streams, monkeypatch):
    made = []
    real = torch.zeros

    def alloc(prob, device):
        made.append(("ws", streams[-1]))
        return object()

    def zeros(*args, **kwargs):
        made.append(("zeros", streams[-1]))
        return real(*args, **kwargs)

    r = Recorder(monkeypatch, streams)
    r.layer.prob = api.make_problem(2, 16, 4, 2, 16, flags=api.FLAG_EXPERT_CAPACITY)
    r.layer.weights["expert_capacity"] = torch.full((4,), -1, dtype=torch.int32)
    monkeypatch.setattr(api, "alloc_backward_workspace", alloc)
    monkeypatch.setattr(api, "moe_layer_backward", lambda *a: None)
    monkeypatch.setattr(api, "moe_balance_update", lambda *a: None)
    r.layer.backward(r.x, r.x, stream=6)
    assert made == [("ws", 6)]
    monkeypatch.setattr(torch, "zeros", zeros)
    r.layer.balance_update(stream=8)
    assert made[1:] == [("zeros", 8)]
    r.layer.balance_update(stream=8)
    assert len(made) == 2 and streams == [1]
