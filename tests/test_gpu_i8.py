"""8-bit rows and products on the GPU against their 64-bit definition
(serving_ref): integers equal, outputs within the counted roundings."""
import pytest
import torch

import serving_ref as ref
from sparse_mixture_experts_04_b200 import api

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i8(shape, g):
    return torch.randint(-127, 128, shape, dtype=torch.int8, generator=g)


def scales(shape, g, k):
    return (torch.rand(shape, generator=g) + 0.5) / (73.0 * k ** 0.5)


# ------------------------------------------------------------------- rows
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (1, 2048), (257, 1040), (5, 8192), (2, 24592), (2400, 64)])
def test_quantize_rows_equals_the_definition(rows, cols, dt):
    g = gen(rows * cols)
    x = torch.randn((rows, cols), generator=g).to(DT[dt])
    q, s = api.quantize_rows(x.cuda())
    wq, ws = ref.quantize(x)
    assert torch.equal(s.cpu().double(), ws)
    assert torch.equal(q.cpu().double(), wq)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1250, 2032), (1250, 4112), (1250, 8208), (640, 528), (311, 1040), (160, 4000),
                                       (70, 16400), (1, 8176), (5000, 1024)])
def test_quantize_rows_for_every_number_of_warps_per_row(rows, cols, dt):
    """Coarse values, so that ties are common; some rows all equal or zero."""
    g = gen(rows + cols)
    x = torch.randint(-64, 65, (rows, cols), generator=g).float() * 0.375
    x[rows // 2] = 0.0
    x[-1] = -2.5
    x = x.to(DT[dt])
    q, s = api.quantize_rows(x.cuda())
    wq, ws = ref.quantize(x)
    assert torch.equal(s.cpu().double(), ws)
    assert torch.equal(q.cpu().double(), wq)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_rows_at_ties_and_extremes(dt):
    t = DT[dt]
    k = torch.arange(-127, 128).float()
    rows = [
        torch.cat([torch.tensor([127.0]), k[:127] + 0.5]),                 # scale 1: every value a tie
        torch.cat([torch.tensor([-254.0]), k[:127] * 2 + 1]),              # scale 2: ties again
        torch.full((128,), 3.0),
        torch.zeros(128),
        torch.full((128,), 1e-44),                                         # subnormal: the scale's floor
        torch.linspace(-1, 1, 128) * 2.0 ** -130,
        torch.linspace(-1, 1, 128) * 3.3e38,
        torch.cat([torch.tensor([1.0]), torch.full((127,), 1e-30)]),
        -torch.linspace(0, 1, 128) ** 8,
    ]
    x = torch.stack(rows).to(t)
    q, s = api.quantize_rows(x.cuda())
    wq, ws = ref.quantize(x)
    assert torch.equal(s.cpu().double(), ws)
    assert torch.equal(q.cpu().double(), wq)


def test_quantize_rows_next_to_ties():
    """Values one unit in the last place around every tie of an odd scale."""
    s = torch.tensor(0.7281937)
    amax = s * 127.0
    ties = (torch.arange(-127, 127).float() + 0.5) * s
    x = torch.cat([torch.tensor([float(amax)]), ties, torch.nextafter(ties, torch.tensor(9e9)),
                   torch.nextafter(ties, torch.tensor(-9e9)), torch.zeros(5)])
    x = torch.cat([x, torch.zeros(-len(x) % 16)]).reshape(1, -1)
    q, sc = api.quantize_rows(x.cuda())
    wq, ws = ref.quantize(x)
    assert torch.equal(sc.cpu().double(), ws) and torch.equal(q.cpu().double(), wq)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_rows_marks_only_the_bad_row(bad):
    x = torch.randn((3, 64), generator=gen(5))
    x[1, 17] = bad
    q, s = api.quantize_rows(x.cuda())
    wq, ws = ref.quantize(x)
    assert torch.equal(q.cpu().double(), wq)
    assert torch.isnan(s[1]) and torch.equal(s.cpu().double()[[0, 2]], ws[[0, 2]])


# ---------------------------------------------------------------- products
def run_matmul(x, xs, off, w, ws, dt, rows, fill=0.0):
    y = torch.full((rows, w.shape[-2]), fill, dtype=dt, device="cuda")
    buf = api.alloc_matmul_workspace()
    api.moe_matmul_i8(x.cuda(), xs.cuda(), None if off is None else off.cuda(), w.cuda(), ws.cuda(), y, buf)
    assert api.read_device_status(buf) == 0
    return y.cpu()


def check_product(y, x, xs, w, ws, dt):
    want = (x.double() @ w.double().T) * (xs.double()[:, None] * ws.double())
    # int32 to FP32, the product of the scales, their product: 3 roundings, and the output's
    bound = (3.01 * ref.U + (HALF[dt] if dt == torch.bfloat16 else 0.0)) * want.abs()
    assert torch.all((y.double() - want).abs() <= bound), (y.double() - want).abs().max()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,N,K", [(1, 8, 16), (1, 2816, 2048), (2, 136, 48), (7, 264, 1040), (16, 512, 4096),
                                      (33, 96, 80), (129, 1416, 1040), (300, 256, 128), (255, 8, 2064),
                                      (513, 392, 528)])
def test_matmul_one_group(rows, N, K, dt):
    g = gen(rows + N + K)
    x, xs, w, ws = i8((rows, K), g), scales((rows,), g, 1), i8((N, K), g), scales((N,), g, K)
    check_product(run_matmul(x, xs, None, w, ws, dt, rows), x, xs, w, ws, dt)


@pytest.mark.parametrize("sizes", [[0, 5, 0, 1, 130, 0], [300, 0, 257, 2, 256], [1] * 40, [0, 0, 3], [700, 33, 64],
                                   [260, 259, 288, 300]])
@pytest.mark.parametrize("K", [256, 272])
def test_matmul_groups_and_rows_of_no_group(sizes, K):
    g = gen(sum(sizes))
    G, N, tail = len(sizes), 392, 9
    off = torch.tensor([0] + sizes).cumsum(0).int()
    rows = int(off[-1]) + tail
    x, xs, w, ws = i8((rows, K), g), scales((rows,), g, 1), i8((G, N, K), g), scales((G, N), g, K)
    y = run_matmul(x, xs, off, w, ws, torch.float32, rows, fill=7.0)
    for i in range(G):
        a, b = int(off[i]), int(off[i + 1])
        if b > a:
            check_product(y[a:b], x[a:b], xs[a:b], w[i], ws[i], torch.float32)
    assert torch.all(y[int(off[-1]):] == 7.0)


def test_matmul_of_extreme_integers_is_exact():
    """-128 and 127 everywhere over the longest tested reduction: the sums pass 2^30."""
    K = 131056
    x = torch.full((2, K), -128, dtype=torch.int8)
    x[1] = 127
    w = torch.full((16, K), -128, dtype=torch.int8)
    w[1::2] = 127
    one = torch.ones(16)
    y = run_matmul(x, one[:2], None, w, one, torch.float32, 2)
    want = (x.double() @ w.double().T).float()
    assert torch.equal(y, want)


# --------------------------------------------------------------------- FFN
def ffn_case(G, sizes, d, F, Ns, seed, tail=0):
    g = gen(seed)
    rows = sum(sizes) + tail
    x = torch.randn((rows, d), generator=g).to(torch.bfloat16)
    c = dict(x=x, off=torch.tensor([0] + sizes).cumsum(0).int(), w13=i8((G, 2 * F, d), g),
             s13=scales((G, 2 * F), g, d), w2=i8((G, d, F), g),
             s2=scales((d,) if Ns else (G, d), g, F * max(Ns, 1)))
    return c


def check_rows(y, q, s, w13, s13, w2, s2):
    want, bound = ref.ffn_i8(q, s, w13, s13, w2, s2)
    err = (y.double() - want).abs()
    assert torch.all(err <= bound * (1 + ref.BF16_HALF) + ref.BF16_HALF * want.abs()), float((err - bound).max())


@pytest.mark.parametrize("sizes,d,F", [([1], 16, 16), ([3, 0, 2], 64, 48), ([40, 200, 1, 0, 90], 144, 80),
                                       ([300, 520, 0, 257], 128, 272), ([2] * 32, 512, 208), ([1024, 33], 256, 256)])
def test_ffn_routed(sizes, d, F):
    c = ffn_case(len(sizes), sizes, d, F, 0, sum(sizes), tail=3)
    rows = c["x"].shape[0]
    prob = api.make_problem(rows, d, len(sizes), 1, F)
    xq, xs = api.quantize_rows(c["x"].cuda())
    y = torch.full((rows, d), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = api.alloc_i8_workspace(prob)
    api.moe_expert_ffn_i8(prob, api.FFN_ROUTED, xq, xs, c["off"].cuda(), c["w13"].cuda(), c["s13"].cuda(),
                          c["w2"].cuda(), c["s2"].cuda(), y, ws)
    assert api.read_device_status(ws) == 0
    q, s = ref.quantize(c["x"])
    for i in range(len(sizes)):
        a, b = int(c["off"][i]), int(c["off"][i + 1])
        if b > a:
            check_rows(y[a:b].cpu(), q[a:b], s[a:b], c["w13"][i], c["s13"][i], c["w2"][i], c["s2"][i])
    assert torch.all(y[int(c["off"][-1]):] == 5.0)


@pytest.mark.parametrize("rows,Ns", [(1, 1), (37, 3), (300, 2), (513, 1)])
def test_ffn_shared_is_one_wide_expert(rows, Ns):
    d, F = 144, 80
    c = ffn_case(Ns, [rows], d, F, Ns, rows)
    prob = api.make_problem(rows, d, 4, 1, F, n_shared=Ns)
    xq, xs = api.quantize_rows(c["x"].cuda())
    y = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    ws = api.alloc_i8_workspace(prob)
    api.moe_expert_ffn_i8(prob, api.FFN_SHARED, xq, xs, None, c["w13"].cuda(), c["s13"].cuda(), c["w2"].cuda(),
                          c["s2"].cuda(), y, ws)
    assert api.read_device_status(ws) == 0
    q, s = ref.quantize(c["x"])
    w13 = torch.cat([c["w13"][:, :F].reshape(Ns * F, d), c["w13"][:, F:].reshape(Ns * F, d)])
    s13 = torch.cat([c["s13"][:, :F].reshape(-1), c["s13"][:, F:].reshape(-1)])
    check_rows(y.cpu(), q, s, w13, s13, c["w2"].permute(1, 0, 2).reshape(d, Ns * F), c["s2"])


def test_ffn_repeats_bit_for_bit_and_keeps_a_bad_row_to_itself():
    sizes, d, F = [290, 70, 5], 256, 144
    c = ffn_case(3, sizes, d, F, 0, 9)
    prob = api.make_problem(sum(sizes), d, 3, 1, F)
    ws = api.alloc_i8_workspace(prob)
    dev = {k: v.cuda() for k, v in c.items()}

    def run(x):
        y = torch.empty_like(x)
        xq, xs = api.quantize_rows(x)
        api.moe_expert_ffn_i8(prob, api.FFN_ROUTED, xq, xs, dev["off"], dev["w13"], dev["s13"], dev["w2"], dev["s2"],
                              y, ws)
        return y

    a = run(dev["x"])
    ws.random_(0, 256)   # scratch: what it holds does not matter
    ws[:256] = 0
    assert torch.equal(a, run(dev["x"]))
    x = dev["x"].clone()
    x[3, 1] = float("nan")
    b = run(x)
    assert torch.isnan(b[3]).all()
    keep = torch.arange(len(x), device="cuda") != 3
    assert torch.equal(a[keep], b[keep])
