"""The serving operators together, as a program uses them: a layer quantised
from its weights, its forward for many tokens and for a few, captured, from host
batches, with capacities that adapt between steps."""
import pytest
import torch

import serving_ref as ref
from sparse_mixture_experts_04_b200 import MoeLayer, MoeLayerI8, api, quantize_weights
from sparse_mixture_experts_04_b200.synth import exact_router_inputs

pytestmark = pytest.mark.gpu


def inputs(T, d, E, K, F, Ns, seed):
    g = torch.Generator().manual_seed(seed)
    inp = exact_router_inputs(T, d, E, seed)
    bf = torch.bfloat16
    inp["w13"] = (torch.randn((E, 2 * F, d), generator=g) / d ** 0.5).to(bf)
    inp["w2"] = (torch.randn((E, d, F), generator=g) / F ** 0.5).to(bf)
    if Ns:
        inp["w13_shared"] = (torch.randn((Ns, 2 * F, d), generator=g) / d ** 0.5).to(bf)
        inp["w2_shared"] = (torch.randn((Ns, d, F), generator=g) / F ** 0.5).to(bf)
    return inp


def layer_of(inp, K, F, Ns, C=0.0, flags=0):
    T, d = inp["x"].shape
    prob = api.make_problem(T, d, inp["w13"].shape[0], K, F, Ns, C, "bf16", flags, 0.01)
    w = {k: torch.as_tensor(v).cuda() for k, v in inp.items() if k != "x"}
    return MoeLayer(prob, w)


def quantised(inp):
    """inp with 8-bit weights by the 64-bit rule (CPU)."""
    out = {k: v for k, v in inp.items()}
    for k in ("w13", "w2", "w13_shared"):
        if k in inp:
            q, s = ref.quantize(inp[k])
            out[k], out[k + "_scale"] = q.to(torch.int8), s.float()
    if "w2_shared" in inp:
        n, d, F = inp["w2_shared"].shape
        q, s = ref.quantize(inp["w2_shared"].permute(1, 0, 2).reshape(d, n * F))
        out["w2_shared"] = q.reshape(d, n, F).permute(1, 0, 2).contiguous().to(torch.int8)
        out["w2_shared_scale"] = s.float()
    return out


def check(y, want, rounded_outputs):
    """rounded_outputs: expert outputs rounded to BF16 before they are added."""
    w = want["y"]
    bound = want["bound"] + 64 * ref.U * want["mag"] + (ref.BF16_HALF * 1.01 * want["mag"] if rounded_outputs else 0.0)
    err = (y.cpu().double() - w).abs()
    assert torch.all(err <= bound * (1 + ref.BF16_HALF) + ref.BF16_HALF * w.abs() + 1e-30), float((err - bound).max())


@pytest.mark.parametrize("Ns", [0, 1, 3])
def test_quantised_weights_equal_the_rule(Ns):
    inp = inputs(4, 96, 5, 2, 48, Ns, 11)
    want = quantised(inp)
    got = quantize_weights({k: torch.as_tensor(v).cuda() for k, v in inp.items() if k != "x"})
    for k in ("w13", "w2") + (("w13_shared", "w2_shared") if Ns else ()):
        assert torch.equal(got[k].cpu(), want[k]), k
        assert torch.equal(got[k + "_scale"].cpu(), want[k + "_scale"]), k
    assert torch.equal(got["w_gate"].cpu(), inp["w_gate"])


@pytest.mark.parametrize("T,d,E,K,F,Ns,C", [(1, 64, 4, 2, 48, 0, 0.0), (40, 96, 6, 2, 80, 2, 1.0),
                                            (300, 128, 8, 2, 144, 1, 1.25), (700, 256, 4, 1, 272, 0, 0.0),
                                            (2500, 64, 3, 1, 48, 1, 0.6)])
def test_layer_forward_i8(T, d, E, K, F, Ns, C):
    inp = inputs(T, d, E, K, F, Ns, T)
    layer = MoeLayerI8.from_layer(layer_of(inp, K, F, Ns, C))
    y = layer.forward(inp["x"].cuda())
    assert api.read_device_status(layer.ws) == 0
    cap = api.capacity(layer.prob)
    want = ref.few_layer(quantised(inp), K, [cap] * E, False)
    for k in ("topk_idx", "counts", "kept", "seg_off", "slot_of"):
        assert torch.equal(layer.routing[k].cpu(), want[k].reshape(layer.routing[k].shape)), k
    check(y, want, True)
    if T <= api.FEW_MAX_TOKENS:
        stats = layer.stats.clone()
        check(layer.forward_few(inp["x"].cuda()), want, False)
        assert torch.allclose(layer.stats, stats, rtol=4e-7, atol=0)


@pytest.mark.parametrize("T,d,Ns,C", [(1250, 2064, 1, 0.5), (200, 4112, 0, 0.0), (90, 8208, 1, 1.0), (70, 16400, 1, 0.7)])
def test_wide_tokens_reach_their_rows(T, d, Ns, C):
    """Tokens that take several warps, or a whole block twice, to round; dropped pairs."""
    inp = inputs(T, 64, 4, 2, 48, Ns, T + d)  # exact logits of 64 values; the rest has no say in the routing
    g = torch.Generator().manual_seed(d)
    for k in [k for k in ("x", "w_gate", "w13", "w13_shared") if k in inp]:
        more = torch.zeros if k == "w_gate" else (lambda s: torch.randn(s, generator=g) * (1 if k == "x" else d ** -0.5))
        t = torch.as_tensor(inp[k])
        inp[k] = torch.cat([t, more((*t.shape[:-1], d - 64)).to(t.dtype)], -1)
    for k in [k for k in ("w2", "w2_shared") if k in inp]:
        inp[k] = (torch.randn((*inp[k].shape[:-2], d, 48), generator=g) / 48 ** 0.5).to(torch.bfloat16)
    layer = MoeLayerI8.from_layer(layer_of(inp, 2, 48, Ns, C))
    y = layer.forward(inp["x"].cuda())
    assert api.read_device_status(layer.ws) == 0
    want = ref.few_layer(quantised(inp), 2, [api.capacity(layer.prob)] * 4, False)
    assert torch.equal(layer.routing["slot_of"].cpu(), want["slot_of"].reshape(T, 2))
    check(y, want, True)


@pytest.mark.parametrize("cls", [MoeLayer, MoeLayerI8])
def test_the_forwards_of_one_layer_agree(cls):
    """forward, forward_few, a captured forward and forward_host of the same
    layer, interleaved; every one repeats bit for bit."""
    T, d, E, K, F, Ns = 24, 128, 8, 2, 96, 1
    inp = inputs(T, d, E, K, F, Ns, 5)
    base = layer_of(inp, K, F, Ns, 1.0)
    layer = base if cls is MoeLayer else MoeLayerI8.from_layer(base)
    want = ref.few_layer(inp if cls is MoeLayer else quantised(inp), K, [api.capacity(base.prob)] * E, cls is MoeLayer)
    x = inp["x"].cuda()
    a, b = layer.forward(x).clone(), layer.forward_few(x).clone()
    check(a, want, True)
    check(b, want, False)
    layer.capture()
    for _ in range(2):
        assert torch.equal(layer.forward_graphed(x), a)
        assert torch.equal(layer.forward_few(x), b)
        assert torch.equal(layer.forward(x), a)
    xs = [inp["x"].pin_memory(), (-inp["x"]).pin_memory(), inp["x"].pin_memory()]
    ys = [torch.empty((T, d), dtype=torch.bfloat16).pin_memory() for _ in xs]
    layer.forward_host(xs, ys)
    assert torch.equal(ys[0], a.cpu()) and torch.equal(ys[2], a.cpu())


def test_decode_steps_with_adaptive_capacities():
    """balance_update between forward_few steps: the next step keeps what the
    updated capacities allow."""
    T, d, E, K, F = 48, 64, 6, 2, 48
    inp = inputs(T, d, E, K, F, 0, 8)
    layer = layer_of(inp, K, F, 0, 1.0, api.FLAG_EXPERT_CAPACITY)
    x = inp["x"].cuda()
    for _ in range(3):
        caps = layer.weights["expert_capacity"].cpu().tolist()
        y = layer.forward_few(x)
        want = ref.few_layer(inp, K, caps, True)
        assert torch.equal(layer.routing["kept"].cpu(), want["kept"])
        assert torch.equal(layer.routing["slot_of"].cpu(), want["slot_of"])
        check(y, want, False)
        layer.balance_update(gamma=0.5, c_base=0.9)
    assert layer.weights["expert_capacity"].cpu().tolist() != [-1] * E


def test_ffn_i8_without_live_rows():
    prob = api.make_problem(40, 64, 4, 1, 48)
    x, s = api.quantize_rows(torch.randn((40, 64), device="cuda").bfloat16())
    g = torch.Generator(device="cuda").manual_seed(1)
    i8 = lambda *sh: torch.randint(-127, 128, sh, dtype=torch.int8, device="cuda", generator=g)
    y = torch.full((40, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = api.alloc_i8_workspace(prob)
    api.moe_expert_ffn_i8(prob, api.FFN_ROUTED, x, s, torch.zeros(5, dtype=torch.int32, device="cuda"), i8(4, 96, 64),
                          torch.ones((4, 96), device="cuda"), i8(4, 64, 48), torch.ones((4, 64), device="cuda"), y, ws)
    assert torch.all(y == 3.0) and api.read_device_status(ws) == 0


def test_binding_refuses_wrong_tensors():
    x = torch.randn((4, 64), device="cuda").bfloat16()
    q, s = api.quantize_rows(x)
    w = torch.zeros((16, 64), dtype=torch.int8, device="cuda")
    ws = api.alloc_matmul_workspace()
    y = torch.empty((4, 16), device="cuda")
    ok = (q, s, None, w, torch.ones(16, device="cuda"), y, ws)
    api.moe_matmul_i8(*ok)
    for i, bad in ((0, q[:, ::2]), (0, q[:, :32].contiguous()), (1, s[:3]), (1, s.double()), (3, w.t()),
                   (4, torch.ones(8, device="cuda")), (5, y.half()), (5, y[:3]), (6, ws.cpu()),
                   (2, torch.zeros(3, dtype=torch.int32, device="cuda"))):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            api.moe_matmul_i8(*args)
    with pytest.raises(ValueError):
        api.moe_quantize_rows(x.half(), q, s)
    with pytest.raises(ValueError):
        api.moe_quantize_rows(x, q, s[:2])
    with pytest.raises(api.MoeError):
        api.quantize_rows(x[:, :8].contiguous())      # not a multiple of 16
    inp = inputs(4, 64, 4, 2, 48, 0, 2)
    layer = layer_of(inp, 2, 48, 0)
    with pytest.raises(ValueError):
        layer.forward_few(inp["x"].cuda()[:3])
    with pytest.raises(ValueError):
        layer.forward_few(inp["x"])
    layer = layer_of(inp, 2, 48, 0)
    layer.weights["w2"] = layer.weights["w2"].float()
    with pytest.raises(ValueError):                   # weights are checked by the first call
        layer.forward_few(inp["x"].cuda())
    with pytest.raises(ValueError):
        MoeLayerI8(layer.prob, layer.weights)
    big = layer_of(inputs(65, 64, 4, 2, 48, 0, 2), 2, 48, 0)
    with pytest.raises(api.MoeError):
        big.forward_few(torch.zeros((65, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(RuntimeError):
        MoeLayerI8.from_layer(big).backward(None, None)
