"""The few-token layer and the 8-bit entry points on the host (no GPU): sizes,
refusals before anything is enqueued, argument checks of the Python binding, and
the 64-bit forms the GPU tests compare with, checked against the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import serving_ref as ref
from sparse_mixture_experts_04_b200 import MoeLayerI8, _lib, api, build
from sparse_mixture_experts_04_b200.synth import exact_router_inputs

FAKE = 4096          # non-null, 256-byte aligned, never dereferenced
WS = 1 << 20


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def weights(**kw):
    w = dict(w_gate=FAKE, logit_offset=None, sel_bias=None, w13=FAKE, w2=FAKE, w13_shared=None, w2_shared=None,
             expert_capacity=None)
    w.update(kw)
    return _lib.MoeWeights(*w.values())


def weights_i8(**kw):
    w = {k: FAKE for k, _ in _lib.MoeWeightsI8._fields_}
    for k in ("logit_offset", "sel_bias", "w13_shared", "w13_shared_scale", "w2_shared", "w2_shared_scale",
              "expert_capacity"):
        w[k] = None
    w.update(kw)
    return _lib.MoeWeightsI8(*w.values())


def size(fn, prob):
    n = ctypes.c_size_t(0)
    return fn(ctypes.byref(prob), ctypes.byref(n)), n.value


# -------------------------------------------------------------------- few tokens
def call_few(L, prob, w=None, x=FAKE, y=FAKE, routing=None, ws=WS, nbytes=None, i8=False):
    n = size(L.moe_few_workspace_size, prob)[1] if nbytes is None else nbytes
    fn = L.moe_layer_forward_few_i8 if i8 else L.moe_layer_forward_few
    w = (weights_i8() if i8 else weights()) if w is None else w
    return fn(ctypes.byref(prob), x, ctypes.byref(w), y, routing, None, ws, n, None)


def test_few_workspace_and_token_limit(L):
    assert api.FEW_MAX_TOKENS == 64
    for T in (1, 64):
        assert size(L.moe_few_workspace_size, api.make_problem(T, 64, 8, 2, 128))[0] == 0
    assert size(L.moe_few_workspace_size, api.make_problem(65, 64, 8, 2, 128))[0] == -2
    big = 1 << 40
    for i8 in (False, True):
        assert call_few(L, api.make_problem(65, 64, 8, 2, 128), nbytes=big, i8=i8) == -2
    # the widest rows: BF16 34784, FP32 17392, 8-bit 69568 columns
    assert call_few(L, api.make_problem(1, 34792, 1, 1, 16), nbytes=big) == -2
    assert call_few(L, api.make_problem(1, 17400, 1, 1, 16, dtype="f32"), nbytes=big) == -2
    assert call_few(L, api.make_problem(1, 69584, 1, 1, 16), nbytes=big, i8=True) == -2
    assert size(L.moe_few_workspace_size, api.make_problem(1, 69568, 1, 1, 16))[0] == 0
    assert size(L.moe_few_workspace_size, api.make_problem(1, 69584, 1, 1, 16))[0] == -2
    with pytest.raises(api.MoeError):
        api.few_workspace_size(api.make_problem(65, 64, 8, 2, 128))


@pytest.mark.parametrize("i8", [False, True])
def test_few_refuses_bad_arguments(L, i8):
    prob = api.make_problem(8, 64, 8, 2, 128)
    W = weights_i8 if i8 else weights
    assert call_few(L, prob, x=None, i8=i8) == -1
    assert call_few(L, prob, x=FAKE + 4, i8=i8) == -1
    assert call_few(L, prob, y=None, i8=i8) == -1
    assert call_few(L, prob, W(w13=None), i8=i8) == -1
    assert call_few(L, prob, W(w2=FAKE + 8), i8=i8) == -1
    assert call_few(L, prob, W(w_gate=None), i8=i8) == -1
    assert call_few(L, prob, W(w13_shared=FAKE, w2_shared=FAKE), i8=i8) == -1      # shared weights, none shared
    assert call_few(L, api.make_problem(8, 64, 8, 2, 128, n_shared=1), i8=i8) == -1
    assert call_few(L, prob, ws=None, i8=i8) == -5
    assert call_few(L, prob, ws=WS + 16, i8=i8) == -5
    assert call_few(L, prob, nbytes=size(L.moe_few_workspace_size, prob)[1] - 1, i8=i8) == -5
    assert call_few(L, api.make_problem(8, 64, 8, 2, 128, flags=api.FLAG_SAVE_GU), i8=i8) == -1
    assert call_few(L, api.make_problem(8, 64, 8, 2, 128, flags=api.FLAG_LOGITS_GIVEN), i8=i8) == -1  # no logits
    cap = api.make_problem(8, 64, 8, 2, 128, flags=api.FLAG_EXPERT_CAPACITY)
    assert call_few(L, cap, i8=i8) == -1
    assert call_few(L, cap, W(expert_capacity=FAKE + 4), i8=i8) == -1


# ----------------------------------------------------------------- 8-bit integers
def test_i8_problems(L):
    assert size(L.moe_i8_workspace_size, api.make_problem(100, 64, 8, 2, 128))[0] == 0
    for bad, code in ((api.make_problem(100, 72, 8, 2, 128), -1), (api.make_problem(100, 64, 8, 2, 136), -1),
                      (api.make_problem(100, 64, 8, 2, 128, dtype="f32"), -2),
                      (api.make_problem(100, 64, 8, 2, 128, flags=api.FLAG_SAVE_GU), -1),
                      (api.make_problem(1, 131072, 1, 1, 16), -2), (api.make_problem(1, 16, 1, 1, 131072), -2),
                      (api.make_problem(1, 16, 1, 1, 65536, n_shared=2), -2)):
        assert size(L.moe_i8_workspace_size, bad)[0] == code
    assert size(L.moe_i8_workspace_size, api.make_problem(1, 131056, 1, 1, 16))[0] == 0


@pytest.mark.parametrize("kw", [dict(n_rows=0), dict(n_rows=-1), dict(n_cols=8), dict(n_cols=24), dict(dtype=2),
                                dict(x=None), dict(x=FAKE + 8), dict(q=None), dict(q=FAKE + 4), dict(s=None),
                                dict(s=FAKE + 4)])
def test_quantize_rows_refusals(L, kw):
    a = dict(n_rows=4, n_cols=32, dtype=0, x=FAKE, q=FAKE, s=FAKE)
    a.update(kw)
    assert L.moe_quantize_rows(a["n_rows"], a["n_cols"], a["dtype"], a["x"], a["q"], a["s"], None) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(G=0), -1), (dict(rows=0), -1), (dict(N=4), -1), (dict(N=12), -1), (dict(K=8), -1), (dict(K=40), -1),
    (dict(out=2), -1), (dict(x=None), -1), (dict(xs=None), -1), (dict(w=FAKE + 8), -1), (dict(ws_=None), -1),
    (dict(y=FAKE + 4), -1), (dict(off=None), -1), (dict(G=257), -2), (dict(K=131072), -2), (dict(rows=1 << 31), -2),
    (dict(N=1 << 30), -2), (dict(ws=None), -5), (dict(ws=WS + 16), -5), (dict(nbytes=255), -5)])
def test_matmul_i8_refusals(L, kw, code):
    a = dict(G=2, rows=4, N=16, K=32, x=FAKE, xs=FAKE, off=FAKE, w=FAKE, ws_=FAKE, out=0, y=FAKE, ws=WS, nbytes=256)
    a.update(kw)
    assert L.moe_matmul_i8(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(mode=2), -1), (dict(x=None), -1), (dict(xs=FAKE + 4), -1), (dict(rows=0), -1), (dict(rows=201), -1),
    (dict(off=None), -1), (dict(w13=None), -1), (dict(s13=None), -1), (dict(w2=FAKE + 2), -1), (dict(s2=None), -1),
    (dict(y=None), -1), (dict(mode=1), -1), (dict(ws=None), -5), (dict(ws=WS + 8), -5), (dict(short=1), -5)])
def test_expert_ffn_i8_refusals(L, kw, code):
    prob = api.make_problem(100, 64, 8, 2, 128)
    n = size(L.moe_i8_workspace_size, prob)[1]
    a = dict(mode=0, x=FAKE, xs=FAKE, rows=8, off=FAKE, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, y=FAKE, ws=WS, short=0)
    a.update(kw)
    short = a.pop("short")
    assert L.moe_expert_ffn_i8(ctypes.byref(prob), *a.values(), n - short, None) == code


def test_layer_forward_i8_refusals(L):
    prob = api.make_problem(100, 64, 8, 2, 128)
    n = size(L.moe_i8_workspace_size, prob)[1]

    def call(p=prob, w=None, x=FAKE, y=FAKE, ws=WS, nbytes=n):
        w = weights_i8() if w is None else w
        return L.moe_layer_forward_i8(ctypes.byref(p), x, ctypes.byref(w), y, None, None, ws, nbytes, None)

    assert call(x=None) == -1 and call(y=FAKE + 8) == -1
    assert call(w=weights_i8(w13_scale=None)) == -1 and call(w=weights_i8(w2_scale=FAKE + 4)) == -1
    assert call(w=weights_i8(w13_shared=FAKE)) == -1
    assert call(ws=None) == -5 and call(nbytes=n - 1) == -5
    assert call(p=api.make_problem(100, 64, 8, 2, 128, dtype="f32")) == -2
    shared = api.make_problem(100, 64, 8, 2, 128, n_shared=1)
    assert call(p=shared, nbytes=1 << 40) == -1


# ------------------------------------------------------------------ Python binding
def test_python_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros((2, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.quantize_rows(x)
    q = torch.zeros((2, 32), dtype=torch.int8)
    with pytest.raises(ValueError):
        api.moe_matmul_i8(q, torch.zeros(2), None, q, torch.zeros(2), torch.zeros((2, 2)), torch.zeros(256))
    prob = api.make_problem(2, 32, 4, 2, 16)
    with pytest.raises(ValueError):
        api.moe_layer_forward_few(prob, x, dict(w13=x, w2=x), x, None, None, x)
    with pytest.raises(ValueError):
        api.moe_expert_ffn_i8(prob, api.FFN_ROUTED, q, torch.zeros(2), None, q, q, q, q, x, x)
    # the checks themselves, on a device index no host tensor has
    for bad in (q.float(), q[:, ::2], q[:1]):
        with pytest.raises(ValueError):
            api._need("q", bad, (2, 32), torch.int8, -1)
    api._need("q", q, (2, 32), torch.int8, -1)


def test_8bit_layer_checks_its_weights():
    prob = api.make_problem(2, 32, 4, 2, 16)
    w = {"w13": torch.zeros((4, 32, 32), dtype=torch.bfloat16)}
    layer = MoeLayerI8.__new__(MoeLayerI8)
    layer.prob, layer.weights, layer.dtype = prob, w, torch.bfloat16
    with pytest.raises(ValueError, match="w13"):
        layer._check_weights()
    with pytest.raises(RuntimeError):
        layer.backward()


# ------------------------------------------------------- the 64-bit reference forms
def test_reference_quantisation():
    x = torch.tensor([[0.0] * 4, [1.0, -0.5, 0.25, 2.0 ** -30], [127.0, 0.5, 1.5, -2.5], [1.0, float("nan"), 0, 0]])
    q, s = ref.quantize(x)
    assert s[0] == 2.0 ** -126 and torch.equal(q[0], torch.zeros(4, dtype=torch.float64))
    assert q[1].tolist() == [127.0, -64.0, 32.0, 0.0]       # 63.5 is a tie between 63 and 64
    assert q[2].tolist() == [127.0, 0.0, 2.0, -2.0]         # ties to even
    assert torch.isnan(s[3]) and torch.equal(q[3], torch.zeros(4, dtype=torch.float64))


@pytest.mark.parametrize("Ns,C", [(0, 0.0), (2, 1.0)])
def test_reference_layer_equals_the_oracle(Ns, C):
    T, d, E, K, F = 24, 32, 6, 2, 40
    g = torch.Generator().manual_seed(3)
    inp = exact_router_inputs(T, d, E, 7)
    inp["x"], inp["w_gate"] = inp["x"].float(), inp["w_gate"].float()
    inp["w13"] = torch.randn((E, 2 * F, d), generator=g)
    inp["w2"] = torch.randn((E, d, F), generator=g)
    if Ns:
        inp["w13_shared"] = torch.randn((Ns, 2 * F, d), generator=g)
        inp["w2_shared"] = torch.randn((Ns, d, F), generator=g)
    cap = oracle.capacity(T, K, E, C)
    want = ref.few_layer(inp, K, [cap] * E, False)
    l64 = oracle.gate_logits(inp["x"].numpy(), inp["w_gate"].numpy(), inp["logit_offset"])
    idx, w, p = oracle.select(l64, K)
    disp = oracle.dispatch(idx, E, cap)
    assert np.array_equal(want["topk_idx"].numpy(), idx)
    assert np.array_equal(want["slot_of"].numpy(), disp["slot_of"])
    y = oracle.layer_rows(inp["x"].numpy(), inp["w13"].numpy(), inp["w2"].numpy(), idx, w, disp["slot_of"],
                          w13_shared=None if not Ns else inp["w13_shared"].numpy(),
                          w2_shared=None if not Ns else inp["w2_shared"].numpy())
    assert np.max(np.abs(want["y"].numpy() - y)) <= 1e-12 * np.max(np.abs(y))
