"""Calls of the serving operators that their documents allow and that are easy to
get wrong: first calls on a side stream, forwards in other orders, sizes at the
limits."""
import importlib.util
import os

import pytest
import torch

import serving_ref as ref
import test_gpu_few
from sparse_mixture_experts_04_b200 import MoeLayer, MoeLayerI8, api
from test_gpu_few import build, make, run
from test_quant_rule_host import rows_of_every_bf16_maximum

pytestmark = pytest.mark.gpu


def busy():
    """Some 20 ms of ordinary work on the current stream."""
    a = torch.randn((4096, 4096), device="cuda")
    for _ in range(20):
        a = a @ a
        a = a / a.norm()
    return a


@pytest.mark.parametrize("kind", ["bf16", "f32", "i8"])
def test_first_few_token_call_on_a_side_stream(kind):
    """The default stream is busy: nothing that the call enqueues may end up there,
    in front of or behind the kernel (the workspace's clearing would)."""
    inp = make(6, 256, 8, 2, 512, 1, kind, 31)
    want = build(inp, 2, Ns=1).forward_few(inp["x"].cuda()).clone()
    layer, x, y = build(inp, 2, Ns=1), inp["x"].cuda(), torch.zeros_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = busy()
    layer.forward_few(x, y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    torch.cuda.synchronize()
    assert bool(layer.few_ws.any())      # not cleared afterwards
    layer.forward_few(x, y)              # then on the default stream, and as a handle
    layer.forward_few(x, y, stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.isfinite(keep).all()


def test_first_few_token_call_on_the_default_streams_handle():
    """The current stream is a busy one of its own; the call names the default stream."""
    inp = make(6, 256, 8, 2, 512, 1, "bf16", 36)
    want = build(inp, 2, Ns=1).forward_few(inp["x"].cuda()).clone()
    layer, x = build(inp, 2, Ns=1), inp["x"].cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        busy()
        y = layer.forward_few(x, stream=torch.cuda.default_stream().cuda_stream)
        torch.cuda.default_stream().synchronize()
        assert torch.equal(y.cpu(), want.cpu())
    torch.cuda.synchronize()
    assert bool(layer.few_ws.any()) and torch.equal(y, want)


def test_new_outputs_on_a_side_stream_keep_their_values():
    """Outputs made by the calls themselves, while the default stream frees and
    takes blocks of the same sizes behind pending work."""
    inp = make(6, 256, 8, 2, 512, 1, "bf16", 32)
    layer, x = build(inp, 2, Ns=1), inp["x"].cuda()
    want, want_fwd, (want_q, want_s) = layer.forward_few(x).clone(), layer.forward(x).clone(), api.quantize_rows(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy()
        for shape, dt in ((x.shape, x.dtype), (x.shape, torch.int8), (x.shape[:1], torch.float32)):
            torch.zeros(shape, dtype=dt, device="cuda")     # enqueued behind the work, and freed at once
        y = layer.forward_few(x, stream=side)
        z = layer.forward(x, stream=side)
        q, s = api.quantize_rows(x, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want_fwd)
        assert torch.equal(q, want_q) and torch.equal(s, want_s)


def test_a_few_token_call_between_forward_and_backward():
    """With routing arrays backward() refuses; without, the pending gradients are
    those of the forward alone, bit for bit."""
    T, d, E, K, F, Ns = 24, 128, 8, 2, 128, 1
    inp = make(T, d, E, K, F, Ns, "bf16", 33)
    x, other = inp["x"].cuda(), inp["x"].flip(0).cuda().contiguous()
    dy = torch.randn((T, d), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = {k: torch.as_tensor(v).cuda() for k, v in inp.items() if k != "x" and v is not None}
    prob = api.make_problem(T, d, E, K, F, Ns, 1.0, "bf16", 0, 0.01)
    plain = MoeLayer(prob, w)
    plain.forward(x)
    want = {k: v.clone() for k, v in plain.backward(x, dy).items()}
    plain.forward_few(other)
    with pytest.raises(RuntimeError):
        plain.backward(x, dy)
    plain.forward(x)
    again = plain.backward(x, dy)
    bare = MoeLayer(prob, w, keep_routing=False)
    bare.forward(x)
    bare.forward_few(other)
    got = bare.backward(x, dy)
    for k, v in want.items():
        assert torch.equal(again[k], v) and torch.equal(got[k], v), k


def test_balance_update_of_the_8bit_layer_leaves_its_source_alone():
    T, E = 48, 6
    inp = make(T, 64, E, 2, 48, 0, "bf16", 34, bias=0.1)
    base = build(inp, 2, 1.0, api.FLAG_EXPERT_CAPACITY)
    small = MoeLayerI8.from_layer(base)
    x = inp["x"].cuda()
    before = {k: base.weights[k].clone() for k in ("sel_bias", "expert_capacity")}
    first = base.forward_few(x).clone()
    for _ in range(2):
        small.forward_few(x)
        small.balance_update(bias_rate=0.05, c_base=0.9, gamma=0.5)
    for k, v in before.items():
        assert torch.equal(base.weights[k], v) and not torch.equal(small.weights[k], v), k
    assert torch.equal(base.forward_few(x), first)


def test_a_training_layer_and_its_8bit_copy():
    """FLAG_SAVE_GU has no meaning for the copy, which equals the one made of the
    same layer without the flag."""
    inp = make(20, 64, 6, 2, 48, 1, "bf16", 35)
    x = inp["x"].cuda()
    a = MoeLayerI8.from_layer(build(inp, 2, 1.0, api.FLAG_SAVE_GU, None, 1))
    b = MoeLayerI8.from_layer(build(inp, 2, 1.0, 0, None, 1))
    assert torch.equal(a.forward(x), b.forward(x)) and torch.equal(a.forward_few(x), b.forward_few(x))
    assert api.read_device_status(a.ws) == 0 and api.read_device_status(a.few_ws) == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_one_scale_rule_everywhere(dt):
    """moe_quantize_rows, the 64-bit form of the tests, elementary torch operations
    on the GPU and the measured cases' plain form: one rule, bit for bit."""
    spec = importlib.util.spec_from_file_location(
        "measured_cases", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py"))
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    x = rows_of_every_bf16_maximum().to(dt).cuda()
    q, s = api.quantize_rows(x)
    wq, ws = ref.quantize(x.cpu())
    assert torch.equal(s.cpu().double(), ws) and torch.equal(q.cpu().double(), wq)
    t = x.float().abs().amax(1) / 127.0
    assert torch.equal(s, t) and torch.equal(q.double(), torch.round(x.double() / t.double()[:, None]))
    pq, ps = cases._quantize(x)
    assert torch.equal(q.float(), pq) and torch.equal(s, ps)


# ------------------------------------------------------------ sizes at the limits
@pytest.fixture
def wide_router(monkeypatch):
    """exact_router_inputs for rows of more than 4096: the columns beyond have no say
    in the routing (gate weights of zero), so the logits stay exact."""
    exact = test_gpu_few.exact_router_inputs

    def inputs(T, d, E, seed):
        inp = exact(T, min(d, 4096), E, seed)
        if d > 4096:
            more = torch.randn((T, d - 4096), generator=torch.Generator().manual_seed(seed + d))
            inp["x"] = torch.cat([inp["x"].float(), more], 1)
            inp["w_gate"] = torch.cat([inp["w_gate"].float(), torch.zeros((E, d - 4096))], 1)
        return inp

    monkeypatch.setattr(test_gpu_few, "exact_router_inputs", inputs)


@pytest.mark.parametrize("T,d,E,K,F,Ns,C", [
    (64, 4096, 2, 1, 4120, 1, 0.0),     # 32 rows per expert: groups of 16, three uneven chunks of the reduction
    (33, 4096, 2, 2, 4104, 0, 0.0),     # groups of 16, 16 and 1
    (48, 2816, 3, 2, 2072, 2, 0.75),    # chunks of one and a half stages, a capacity
    (61, 6144, 2, 1, 2056, 1, 0.0),
    (60, 4096, 3, 2, 2072, 2, 0.75),
])
def test_few_layer_of_wide_rows_and_many_tokens(T, d, E, K, F, Ns, C, wide_router):
    """BF16 rows of more than 4 KB with more than 8 rows per expert (token groups
    of up to 16 rows, 32 with the hidden rows' low parts)."""
    run(T, d, E, K, F, Ns, "bf16", C)


@pytest.mark.parametrize("kind,d", [("bf16", 34784), ("f32", 17392), ("i8", 69568)])
@pytest.mark.parametrize("T", [1, 5])
def test_few_layer_of_the_widest_rows(T, kind, d, wide_router):
    run(T, d, 2, 1, 16, 1, kind)


@pytest.mark.parametrize("kind,F", [("bf16", 40008), ("f32", 20008), ("i8", 69584)])
def test_few_layer_of_long_reductions(kind, F):
    """Down products of ten chunks and more."""
    run(5, 64, 2, 1, F, 1, kind)


def quantize_check(x, q, s):
    """Rows against elementary operations on the GPU, a few at a time."""
    inv = torch.tensor(1.0 / 127.0, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // x.shape[1])
    for a in range(0, len(x), step):
        v = x[a:a + step]
        t = (v.float().abs().amax(1) * inv).clamp_(min=2.0 ** -126)
        assert torch.equal(s[a:a + step], t), a
        assert torch.equal(q[a:a + step].double(), torch.round(v.double() / t.double()[:, None])), a


@pytest.mark.parametrize("rows,cols,dt", [
    (524288 + 777, 16, torch.bfloat16), (262144 + 333, 2064, torch.bfloat16), (131072 + 333, 4112, torch.bfloat16),
    (65536 + 333, 8208, torch.bfloat16), (65536 + 33, 16400, torch.bfloat16), (262144 + 333, 1040, torch.float32)])
def test_quantize_more_rows_than_a_grid_holds(rows, cols, dt):
    """One, two, four and eight warps per row and a block per row, more than once around."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.empty((rows, cols), dtype=dt, device="cuda").normal_(generator=g)
    x *= torch.rand((rows, 1), device="cuda", generator=g).to(dt) + 0.01   # neighbours have other maxima
    quantize_check(x, *api.quantize_rows(x))


@pytest.mark.parametrize("T,d,Ns", [(524288 + 777, 64, 1), (262144 + 333, 2064, 0)])
def test_8bit_layer_of_more_tokens_than_a_grid_holds(T, d, Ns):
    """Every token's output equals the one that a layer of its own gives, bit for
    bit: integer sums are exact, and the roundings do not depend on the tile."""
    E, K, F = 4, 2, 16
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *sh: torch.empty(sh, device="cuda").normal_(generator=g)
    i8 = lambda *sh: torch.randint(-127, 128, sh, dtype=torch.int8, device="cuda", generator=g)
    w = dict(w13=i8(E, 2 * F, d), w13_scale=rnd(E, 2 * F).abs() / d, w2=i8(E, d, F), w2_scale=rnd(E, d).abs() / F)
    if Ns:
        w.update(w13_shared=i8(Ns, 2 * F, d), w13_shared_scale=rnd(Ns, 2 * F).abs() / d, w2_shared=i8(Ns, d, F),
                 w2_shared_scale=rnd(d).abs() / F)
    x, logits = rnd(T, d).bfloat16(), rnd(T, E)

    def forward(a, b):
        layer = MoeLayerI8(api.make_problem(b - a, d, E, K, F, Ns, flags=api.FLAG_LOGITS_GIVEN), w)
        layer.routing["logits"].copy_(logits[a:b])
        y = layer.forward(x[a:b], with_stats=False)
        assert api.read_device_status(layer.ws) == 0
        return y

    y = forward(0, T)
    for a in (0, T // 2, T - 900):
        assert torch.equal(y[a:a + 900], forward(a, a + 900)), a
