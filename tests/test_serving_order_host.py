"""Calls of one layer in an order that would mix two forwards' results, refused
or kept apart (no GPU: the entry points are stand-ins)."""
import pytest
import torch

import serving_ref as ref
from sparse_mixture_experts_04_b200 import MoeLayer, MoeLayerI8, api, quantize_weights


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


# ------------------------------------------------------- a layer and its 8-bit copy
@pytest.fixture
def quantisable(monkeypatch):
    """quantize_weights and MoeLayerI8 on CPU tensors, with the 64-bit rule."""
    monkeypatch.setattr(api, "quantize_rows", lambda x: (lambda q, s: (q.to(torch.int8), s.float()))(*ref.quantize(x)))
    monkeypatch.setattr(MoeLayerI8, "_check_weights", lambda self: None)
    g = torch.Generator().manual_seed(2)
    bf = lambda *shape: torch.randn(shape, generator=g).bfloat16()
    return dict(w_gate=bf(4, 16), w13=bf(4, 32, 16), w2=bf(4, 16, 16), sel_bias=torch.zeros(4), logit_offset=None)


def test_the_8bit_layer_adapts_on_its_own(quantisable):
    base = MoeLayer(api.make_problem(2, 16, 4, 2, 16, 0, 1.0, flags=api.FLAG_EXPERT_CAPACITY), quantisable, "cpu")
    small = MoeLayerI8.from_layer(base)
    for k in ("sel_bias", "expert_capacity"):
        assert torch.equal(small.weights[k], base.weights[k])
        before = base.weights[k].clone()
        small.weights[k].add_(1)          # as balance_update does, in place
        assert torch.equal(base.weights[k], before), k
        base.weights[k].sub_(1)
        assert torch.equal(small.weights[k], before + 1), k
    assert quantize_weights({k: v for k, v in quantisable.items() if k != "sel_bias"})["sel_bias"] is None


def test_a_training_layer_can_be_quantised(quantisable):
    flags = api.FLAG_SAVE_GU | api.FLAG_EXTENDED_STATS
    base = MoeLayer(api.make_problem(2, 16, 4, 2, 16, flags=flags), quantisable, "cpu")
    small = MoeLayerI8.from_layer(base)
    assert small.prob.flags == api.FLAG_EXTENDED_STATS and base.prob.flags == flags
    assert small.stats.shape == base.stats.shape


# ------------------------------------------------------------------------ devices
class OnDevice:
    """A contiguous CUDA tensor as far as a check of its properties goes."""
    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.device = shape, dtype, torch.device("cuda", index)

    def is_contiguous(self):
        return True


@pytest.mark.parametrize("cls", [MoeLayer, MoeLayerI8])
def test_weights_on_another_device_are_refused(cls):
    layer = cls.__new__(cls)
    layer.prob, layer.dtype = api.make_problem(2, 32, 4, 2, 16, 1), torch.bfloat16
    layer.ws = OnDevice((1,), torch.uint8, 1)
    good = {k: OnDevice(shape, dtype, 1) for k, (shape, dtype) in layer._weight_shapes().items()}
    good["sel_bias"] = OnDevice((4,), torch.float32, 1)
    layer.weights = good
    layer._check_weights()
    for k, t in good.items():
        layer.weights = dict(good, **{k: OnDevice(t.shape, t.dtype, 0)})
        with pytest.raises(ValueError, match=k):
            layer._check_weights()
