"""The few-token layer (one kernel) against its 64-bit definition (serving_ref):
routing equal (router inputs whose logits are exact), outputs within the counted
roundings, for every weight type, odd sizes, capacities and flags."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from sparse_mixture_experts_04_b200 import MoeLayer, MoeLayerI8, api
from sparse_mixture_experts_04_b200.synth import exact_router_inputs

pytestmark = pytest.mark.gpu


def make(T, d, E, K, F, Ns=0, kind="bf16", seed=0, offset=True, bias=0.0):
    g = torch.Generator().manual_seed(seed * 1000 + T * 7 + d + E + F)
    act = torch.float32 if kind == "f32" else torch.bfloat16
    inp = exact_router_inputs(T, d, E, seed)
    inp["x"], inp["w_gate"] = inp["x"].to(act), inp["w_gate"].to(act)
    if not offset:
        inp["logit_offset"] = None
    inp["sel_bias"] = None
    if bias:
        inp["sel_bias"] = ((torch.rand(E, generator=g) * 2 - 1) * bias).numpy()

    def mat(shape, k):
        if kind == "i8":
            return torch.randint(-127, 128, shape, dtype=torch.int8, generator=g)
        return (torch.randn(shape, generator=g) / k ** 0.5).to(act)

    def sc(shape, k):
        return (torch.rand(shape, generator=g) + 0.5) / (20.0 * k ** 0.5)

    inp["w13"], inp["w2"] = mat((E, 2 * F, d), d), mat((E, d, F), F)
    if Ns:
        inp["w13_shared"], inp["w2_shared"] = mat((Ns, 2 * F, d), d), mat((Ns, d, F), F)
    if kind == "i8":
        inp["w13_scale"], inp["w2_scale"] = sc((E, 2 * F), d), sc((E, d), F)
        if Ns:
            inp["w13_shared_scale"], inp["w2_shared_scale"] = sc((Ns, 2 * F), d), sc((d,), F * Ns)
    return inp


def build(inp, K, C=0.0, flags=0, caps=None, Ns=0, device="cuda"):
    T, d = inp["x"].shape
    E, F2, _ = inp["w13"].shape
    i8 = inp["w13"].dtype == torch.int8
    prob = api.make_problem(T, d, E, K, F2 // 2, Ns, C, "f32" if inp["x"].dtype == torch.float32 else "bf16", flags,
                            0.01)
    w = {k: (None if v is None else torch.as_tensor(v).to(device)) for k, v in inp.items() if k != "x"}
    if caps is not None:
        w["expert_capacity"] = torch.tensor(caps, dtype=torch.int32, device=device)
    return (MoeLayerI8 if i8 else MoeLayer)(prob, w, device)


def limits(T, E, K, C):
    return [-1] * E if C <= 0 else [int(np.ceil(C * (T * K) / E))] * E


def check(layer, y, want, act):
    assert api.read_device_status(layer.few_ws) == 0
    r = layer.routing
    for k in ("topk_idx", "counts", "kept", "seg_off", "slot_of"):
        assert torch.equal(r[k].cpu(), want[k].reshape(r[k].shape)), k
    assert torch.equal(r["logits"].cpu().double(), want["logits"])
    # gates: exp and the sum in FP32, K + 4 roundings and expf's 2 ulp, twice
    assert torch.all((r["topk_w"].cpu().double() - want["topk_w"]).abs() <= (want["topk_w"].shape[1] + 16) * ref.U)
    n = int(want["seg_off"][-1])
    perm, slot = r["perm"].cpu(), want["slot_of"].flatten()
    for i, s in enumerate(slot.tolist()):
        if s >= 0:
            assert int(perm[s]) == i
    assert sorted(perm[:n].tolist()) == [i for i, s in enumerate(slot.tolist()) if s >= 0]
    # the gates' own error on top of the experts' bound
    bound = want["bound"] + 32 * ref.U * want["y"].abs() + want["gate_slack"]
    half = ref.BF16_HALF if act == torch.bfloat16 else ref.U
    err = (y.cpu().double() - want["y"]).abs()
    assert torch.all(err <= bound * (1 + half) + half * want["y"].abs() + 1e-30), float((err - bound).max())


def run(T, d, E, K, F, Ns=0, kind="bf16", C=0.0, flags=0, caps=None, seed=0, bias=0.0):
    inp = make(T, d, E, K, F, Ns, kind, seed, bias=bias)
    layer = build(inp, K, C, flags, caps, Ns)
    x = inp["x"].cuda()
    y = layer.forward_few(x)
    want = ref.few_layer(inp, K, caps if caps is not None else limits(T, E, K, C), kind == "bf16" and "pair",
                         bool(flags & api.FLAG_BIAS_LOGIT))
    # |w error| <= (K + 16) u on each expert's output: bounded by the sum of their magnitudes
    want["gate_slack"] = (K + 16) * ref.U * K * want["y"].abs().amax() * torch.ones_like(want["y"])
    check(layer, y, want, inp["x"].dtype)
    return layer, x, y, want


SIZES = [
    # T, d, E, K, F, Ns, C
    (1, 16, 1, 1, 16, 0, 0.0),
    (1, 64, 4, 1, 64, 0, 0.0),
    (1, 2048, 8, 2, 272, 1, 0.0),
    (2, 80, 4, 4, 48, 0, 1.0),
    (5, 144, 8, 2, 80, 1, 1.0),
    (7, 1040, 16, 4, 528, 2, 1.25),
    (8, 256, 8, 2, 4112, 0, 0.0),       # the down product's reduction in several chunks
    (17, 4096, 4, 2, 64, 0, 0.0),       # several token groups of an expert
    (33, 208, 3, 1, 112, 1, 0.0),       # groups of 9..16 tokens: the second token tile
    (64, 256, 8, 2, 192, 4, 0.0),
    (64, 64, 256, 32, 32, 0, 1.25),     # the most pairs
    (61, 128, 64, 4, 96, 0, 0.5),
]


@pytest.mark.parametrize("kind", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("T,d,E,K,F,Ns,C", SIZES)
def test_few_layer(T, d, E, K, F, Ns, C, kind):
    run(T, d, E, K, F, Ns, kind, C)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d,F", [(8, 8), (24, 40), (72, 88), (1000, 264), (2056, 24), (40, 4104)])
def test_few_layer_multiples_of_eight(d, F, kind):
    run(9, d, 4, 2, F, 1, kind)


@pytest.mark.parametrize("kind", ["bf16", "i8"])
@pytest.mark.parametrize("flags", [0, api.FLAG_BIAS_LOGIT])
def test_few_layer_with_a_selection_bias(flags, kind):
    run(40, 64, 24, 3, 32, 0, kind, 1.0, flags, bias=0.3)


@pytest.mark.parametrize("kind", ["bf16", "f32", "i8"])
def test_few_layer_with_expert_capacities(kind):
    """Zero, one and no limit: tokens that keep nothing get the shared experts only."""
    T, E = 24, 6
    caps = [0, 1, -1, 3, 0, 2]
    run(T, 96, E, 2, 48, 1, kind, 0.0, api.FLAG_EXPERT_CAPACITY, caps)
    layer, x, y, want = run(T, 96, E, 2, 48, 0, kind, 0.0, api.FLAG_EXPERT_CAPACITY, [0] * E)
    assert torch.all(y == 0) and int(want["seg_off"][-1]) == 0


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_few_layer_given_logits(kind):
    T, E, K = 12, 40, 5
    inp = make(T, 64, E, K, 48, 0, kind, 3)
    layer = build(inp, K, 0.0, api.FLAG_LOGITS_GIVEN)
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(4))
    logits[3] = 0.25                      # every expert ties
    logits[4, :20] = -torch.inf           # experts that cannot be chosen by this token
    logits[5, 1:] = -3e38
    layer.routing["logits"].copy_(logits)
    y = layer.forward_few(inp["x"].cuda())
    want = ref.few_layer(inp, K, [-1] * E, kind == "bf16" and "pair", logits=logits.double())
    want["gate_slack"] = (K + 16) * ref.U * K * want["y"].abs().amax() * torch.ones_like(want["y"])
    check(layer, y, want, inp["x"].dtype)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_few_layer_statistics_equal_the_layer_forward(kind):
    """Same statistics as forward(): counts exactly, sums of probabilities to
    their rounding (fixed point, 2^-40 per term, and float32 results)."""
    inp = make(48, 64, 16, 3, 32, 1, kind, 5)
    layer = build(inp, 3, 1.0, api.FLAG_EXTENDED_STATS, None, 1)
    x = inp["x"].cuda()
    layer.forward(x)
    a = layer.stats.clone()
    routing = {k: v.clone() for k, v in layer.routing.items()}
    layer.stats.fill_(-1)
    layer.forward_few(x)
    b = layer.stats
    E = 16
    assert torch.equal(a[:E], b[:E])
    assert torch.allclose(a[E:2 * E + 1], b[E:2 * E + 1], rtol=4e-7, atol=0)
    assert torch.allclose(a[2 * E + 1:], b[2 * E + 1:], rtol=1e-6, atol=0)
    n = int(routing["seg_off"][-1])
    for k, v in routing.items():
        if k == "perm":
            assert torch.equal(v[:n], layer.routing[k][:n])
        elif k != "topk_w":
            assert torch.equal(v, layer.routing[k]), k
    assert torch.allclose(routing["topk_w"], layer.routing["topk_w"], rtol=4e-7, atol=0)


def test_few_layer_repeats_and_ignores_its_workspace_contents():
    layer, x, y, _ = run(30, 512, 16, 4, 256, 1, "bf16")
    first = y.clone()
    layer.few_ws.random_(0, 256)
    for _ in range(3):
        assert torch.equal(layer.forward_few(x), first)
    assert api.read_device_status(layer.few_ws) == 0


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_few_layer_captured_and_replayed(kind):
    inp = make(6, 256, 8, 2, 128, 1, kind, 6)
    layer = build(inp, 2, 0.0, 0, None, 1)
    x, y = inp["x"].cuda(), torch.empty(6, 256, dtype=torch.bfloat16, device="cuda")
    xs = [x, -x, x.flip(0), x * 0.5]
    wants = [layer.forward_few(v).clone() for v in xs]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    buf = torch.empty_like(x)
    with torch.cuda.graph(g):
        layer.forward_few(buf, y)
    for i in (2, 0, 3, 1, 1):
        buf.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wants[i])


def test_few_layer_on_a_side_stream_and_two_layers_at_once():
    a = build(make(4, 256, 8, 2, 512, 0, "bf16", 7), 2)
    b = build(make(4, 256, 8, 2, 512, 0, "bf16", 8), 2)
    xa, xb = make(4, 256, 8, 2, 512, 0, "bf16", 7)["x"].cuda(), make(4, 256, 8, 2, 512, 0, "bf16", 8)["x"].cuda()
    wa, wb = a.forward_few(xa).clone(), b.forward_few(xb).clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ya, yb = torch.empty_like(wa), torch.empty_like(wb)
    for _ in range(20):
        a.forward_few(xa, ya, stream=s1)
        b.forward_few(xb, yb, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(ya, wa) and torch.equal(yb, wb)


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_few_layer_keeps_a_bad_token_to_itself(kind):
    inp = make(5, 64, 4, 2, 32, 1, kind, 9)
    layer = build(inp, 2, 0.0, api.FLAG_LOGITS_GIVEN, None, 1)
    layer.routing["logits"].copy_(torch.randn((5, 4), generator=torch.Generator().manual_seed(1)))
    x = inp["x"].cuda()
    good = layer.forward_few(x).clone()
    x[2, 3] = float("inf")
    bad = layer.forward_few(x)
    assert not torch.isfinite(bad[2]).any() if kind == "i8" else not torch.isfinite(bad[2]).all()
    keep = [0, 1, 3, 4]
    assert torch.equal(good[keep], bad[keep])
