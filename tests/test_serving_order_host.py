"""Calls of one layer in an order that would mix two forwards' results, refused
or kept apart (no GPU: the entry points are stand-ins)."""
import pytest
import torch

from sparse_mixture_experts_04_b200 import MoeLayer, api


@pytest.fixture
def layer(monkeypatch):
    def make(keep_routing):
        layer = MoeLayer(api.make_problem(2, 16, 4, 2, 16), {"w13": None, "w2": None}, "cpu", keep_routing)
        layer._check_weights = lambda: None
        layer._forward = lambda *a: None
        layer._forward_few = lambda *a: None
        return layer

    monkeypatch.setattr(api, "_cuda", lambda name, t: 0)
    monkeypatch.setattr(api, "_current_stream", lambda dev: 1)
    monkeypatch.setattr(api, "alloc_few_workspace", lambda prob, device: object())
    monkeypatch.setattr(api, "alloc_backward_workspace", lambda prob, device: object())
    monkeypatch.setattr(api, "moe_layer_backward", lambda *a: None)
    return make


X = torch.zeros((2, 16), dtype=torch.bfloat16)


def test_backward_refuses_the_routing_of_a_few_token_call(layer):
    m = layer(True)
    m.forward_few(X)
    with pytest.raises(RuntimeError, match="forward_few"):
        m.backward(X, X)                 # no forward at all
    m.forward(X)
    m.backward(X, X)
    m.forward_few(X)
    with pytest.raises(RuntimeError, match="forward_few"):
        m.backward(X, X)                 # the forward's routing is gone
    m.forward(X)
    m.backward(X, X)
    m.backward(X, X)


def test_without_routing_arrays_a_pending_backward_stays_good(layer):
    m = layer(False)
    m.forward_few(X)
    with pytest.raises(RuntimeError, match="forward_few"):
        m.backward(X, X)                 # no forward yet
    m.forward(X)
    m.forward_few(X)
    m.backward(X, X)


def test_a_replayed_forward_counts_as_one(layer):
    m = layer(True)

    class Graph:
        def replay(self):
            pass

    m._graph, m.graph_y = Graph(), X
    m.forward_few(X)
    m.forward_graphed()
    m.backward(X, X)
