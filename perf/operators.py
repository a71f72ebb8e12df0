"""The serving operators of the layer, as measured cases: the whole layer for a
few tokens, the expert FFNs in 8-bit integers and the 8-bit matrix product.

Three operators, told apart by a case's "op":

  few     one layer forward for 1 to 64 tokens (MoeLayer.forward_few, or
          MoeLayerI8.forward_few where "weights" is "i8"): router, capacity,
          routed and shared SwiGLU experts, combine and statistics
  ffn     rows quantised per token, then the grouped SwiGLU experts on 8-bit
          integers with a scale for each token and each output channel
  linear  rows quantised per token, then one grouped matrix product on 8-bit
          integers with the same scales

Quantisation of a row v: s = max(fl32(max|v| / 127), 2^-126), q = the integer
nearest to v / s (ties to even).  A product of 8-bit rows and weights is the
exact integer sum, times the token's scale, times the channel's.
"""
import math

import torch

own = False

FEW_MAX_TOKENS = 64
ALPHA = 0.01


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One token of the fine-grained layer: nothing to share, every microsecond of latency counts.
        dict(name="few_one_fine", op="few", T=1, d=2048, E=128, K=8, F=1024, Ns=4, C=0.0, dtype="bf16",
             weights="bf16", bias=0.1, zipf=0.0),
        # One token through two very wide experts: a stream of 0.7 GB of weights.
        dict(name="few_one_wide", op="few", T=1, d=4096, E=8, K=2, F=14336, Ns=0, C=0.0, dtype="bf16",
             weights="bf16", bias=0.0, zipf=0.0),
        # The decode step of a served batch: 32 tokens touch nearly every expert once or twice.
        dict(name="few_decode", op="few", T=32, d=4096, E=128, K=8, F=1536, Ns=1, C=0.0, dtype="bf16",
             weights="bf16", bias=0.0, zipf=0.0),
        # The same layer with 8-bit experts and a small odd batch under a capacity limit.
        dict(name="few_decode_i8", op="few", T=7, d=4096, E=128, K=8, F=1536, Ns=1, C=1.25, dtype="bf16",
             weights="i8", bias=0.0, zipf=0.0),
        # The most tokens but three on a skewed load: popular experts hold dozens of rows and drop the rest.
        dict(name="few_skewed", op="few", T=61, d=2048, E=64, K=4, F=1408, Ns=0, C=1.0, dtype="bf16",
             weights="bf16", bias=0.0, zipf=1.2),
        # The tiny FP32 layer: no work to speak of, the cost is launches and waits.
        dict(name="few_tiny_f32", op="few", T=64, d=64, E=8, K=2, F=128, Ns=0, C=0.0, dtype="f32",
             weights="f32", bias=0.0, zipf=0.0),
        # Expert FFNs of a decode step on an expert-grouped buffer: two rows per expert, bound by the weights.
        dict(name="ffn_decode", op="ffn", rows=256, tail=0, G=128, d=4096, F=1536, skew=0.0),
        # An ordinary uneven batch: empty experts, part tiles, allocated rows behind the last segment.
        dict(name="ffn_ragged", op="ffn", rows=4901, tail=102, G=64, d=2048, F=1408, skew=1.2),
        # A training-sized batch through eight wide experts: bound by the tensor cores.
        dict(name="ffn_wide", op="ffn", rows=8192, tail=0, G=8, d=4096, F=14336, skew=0.0),
        # One token through one projection: the smallest call there is.
        dict(name="linear_one", op="linear", rows=1, G=1, K=2048, N=2816, dtype="bf16", skew=0.0),
        # Odd sizes in FP32: reduction and columns that end inside every tile, uneven groups.
        dict(name="linear_odd_f32", op="linear", rows=1003, G=9, K=1040, N=1416, dtype="f32", skew=0.8),
        # The skewed layer's up projection over its whole batch of (token, expert) pairs.
        dict(name="linear_pairs", op="linear", rows=65536, G=64, K=2048, N=2816, dtype="bf16", skew=0.5),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    while True:
        op = rng.choice(["few", "few", "ffn", "linear"])
        if op == "few":
            w = rng.choice(["bf16", "bf16", "i8", "f32"])
            step = 16 if w == "i8" else 8
            E = _log_int(rng, 2, 256)
            c = dict(op="few", T=_log_int(rng, 1, FEW_MAX_TOKENS), d=_log_int(rng, 64, 6144, step), E=E,
                     K=rng.randint(1, min(E, 8)), F=_log_int(rng, 64, 8192, step), Ns=rng.choice([0, 0, 1, 2, 4]),
                     C=rng.choice([0.0, 0.0, 1.0, 1.25]), dtype="f32" if w == "f32" else "bf16", weights=w,
                     bias=rng.choice([0.0, 0.0, 0.1]), zipf=rng.choice([0.0, 0.0, 1.2]))
            if 3.0 * (E + c["Ns"]) * c["F"] * c["d"] <= (6e8 if w == "f32" else 2.4e9):
                return c
        elif op == "ffn":
            c = dict(op="ffn", rows=_log_int(rng, 1, 16384), tail=rng.choice([0, 0, rng.randint(1, 200)]),
                     G=_log_int(rng, 1, 128), d=_log_int(rng, 64, 6144, 16), F=_log_int(rng, 64, 8192, 16),
                     skew=rng.choice([0.0, 0.6, 1.2]))
            if 3.0 * c["G"] * c["F"] * c["d"] <= 2.4e9 and 6.0 * c["rows"] * c["F"] * c["d"] <= 1.4e12:
                return c
        else:
            c = dict(op="linear", rows=_log_int(rng, 1, 65536), G=_log_int(rng, 1, 64), K=_log_int(rng, 64, 8192, 16),
                     N=_log_int(rng, 64, 8192, 8), dtype=rng.choice(["bf16", "bf16", "f32"]),
                     skew=rng.choice([0.0, 0.6, 1.2]))
            if 1.0 * c["G"] * c["N"] * c["K"] <= 1e9 and 2.0 * c["rows"] * c["N"] * c["K"] <= 7e11 \
                    and c["rows"] * max(c["N"], c["K"]) <= 2e8:
                return c


# ------------------------------------------------------------------ inputs
def _tdt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _segments(rows, groups, skew, seed):
    """Uneven group sizes: shares ~ rank^-skew in a random order, with a random
    draw of the rows, so that small groups come out empty at times."""
    g = torch.Generator().manual_seed(seed * 7 + 5)
    share = (torch.randperm(groups, generator=g) + 1).double() ** -skew
    pick = torch.multinomial(share, rows, replacement=True, generator=g)
    off = torch.zeros(groups + 1, dtype=torch.int64)
    off[1:] = torch.bincount(pick, minlength=groups).cumsum(0)
    return off.to(torch.int32)


def _i8_rows(shape, g):
    """8-bit weights as a quantised normal matrix has them: the row's largest
    entry, near 4 standard deviations, is 127."""
    q = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in q.view(-1).split(1 << 27):
        part.copy_(torch.empty(part.shape, device="cuda").normal_(0, 31, generator=g).round_().clamp_(-127, 127))
    return q


def _i8_scales(shape, k, g):
    return torch.empty(shape, device="cuda").uniform_(0.9, 1.1, generator=g) / (31.0 * math.sqrt(k))


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std, dt):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(0, std, generator=g)

    if case["op"] == "linear":
        rows, G, K, N = case["rows"], case["G"], case["K"], case["N"]
        return dict(x=normal((rows, K), 1.0, _tdt(case["dtype"])), w=_i8_rows((G, N, K), g),
                    w_scale=_i8_scales((G, N), K, g),
                    seg_off=_segments(rows, G, case["skew"], seed).cuda())
    if case["op"] == "ffn":
        rows, G, d, F = case["rows"], case["G"], case["d"], case["F"]
        return dict(x=normal((rows + case["tail"], d), 1.0, torch.bfloat16), w13=_i8_rows((G, 2 * F, d), g),
                    w13_scale=_i8_scales((G, 2 * F), d, g), w2=_i8_rows((G, d, F), g),
                    w2_scale=_i8_scales((G, d), F, g), seg_off=_segments(rows, G, case["skew"], seed).cuda())
    T, d, E, F, Ns = case["T"], case["d"], case["E"], case["F"], case["Ns"]
    dt = _tdt(case["dtype"])
    s = dict(x=normal((T, d), 1.0, dt), w_gate=normal((E, d), d ** -0.5, dt), sel_bias=None, logit_offset=None)
    if case["weights"] == "i8":
        s["w13"], s["w13_scale"] = _i8_rows((E, 2 * F, d), g), _i8_scales((E, 2 * F), d, g)
        s["w2"], s["w2_scale"] = _i8_rows((E, d, F), g), _i8_scales((E, d), F, g)
        if Ns:
            s["w13_shared"], s["w13_shared_scale"] = _i8_rows((Ns, 2 * F, d), g), _i8_scales((Ns, 2 * F), d, g)
            s["w2_shared"], s["w2_shared_scale"] = _i8_rows((Ns, d, F), g), _i8_scales((d,), F, g)
    else:
        s["w13"], s["w2"] = normal((E, 2 * F, d), d ** -0.5, dt), normal((E, d, F), F ** -0.5, dt)
        if Ns:
            s["w13_shared"] = normal((Ns, 2 * F, d), d ** -0.5, dt)
            s["w2_shared"] = normal((Ns, d, F), F ** -0.5, dt)
    if case["bias"] > 0:
        s["sel_bias"] = torch.empty(E, device="cuda").uniform_(-case["bias"], case["bias"], generator=g)
    if case["zipf"] > 0:
        rank = torch.randperm(E, device="cuda", generator=g) + 1
        s["logit_offset"] = -case["zipf"] * torch.log(rank.float())
    return s


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if not own:
        return s
    from sparse_mixture_experts_04_b200 import MoeLayer, MoeLayerI8, api
    if case["op"] == "few":
        prob = api.make_problem(case["T"], case["d"], case["E"], case["K"], case["F"], case["Ns"], case["C"],
                                case["dtype"], 0, ALPHA)
        weights = {k: v for k, v in s.items() if k not in ("x", "case")}
        s["layer"] = (MoeLayerI8 if case["weights"] == "i8" else MoeLayer)(prob, weights)
        s["y"] = torch.empty_like(s["x"])
        return s
    x = s["x"]
    s["x_q"] = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s["x_scale"] = torch.empty(x.shape[0], device="cuda")
    if case["op"] == "linear":
        s["y"] = torch.zeros((x.shape[0], case["N"]), dtype=x.dtype, device="cuda")
        s["ws"] = api.alloc_matmul_workspace()
    else:
        s["prob"] = api.make_problem(x.shape[0], case["d"], case["G"], 1, case["F"])
        s["y"] = torch.zeros_like(x)
        s["ws"] = api.alloc_i8_workspace(s["prob"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"few": _plain_few, "ffn": _plain_ffn, "linear": _plain_linear}[op](s)
    from sparse_mixture_experts_04_b200 import api
    if op == "few":
        layer = s["layer"]
        layer.forward_few(s["x"], s["y"])
        r = layer.routing
        return dict(y=s["y"], logits=r["logits"], topk_idx=r["topk_idx"], topk_w=r["topk_w"], counts=r["counts"],
                    slot_of=r["slot_of"], stats=layer.stats)
    api.moe_quantize_rows(s["x"], s["x_q"], s["x_scale"])
    if op == "linear":
        api.moe_matmul_i8(s["x_q"], s["x_scale"], s["seg_off"], s["w"], s["w_scale"], s["y"], s["ws"])
    else:
        api.moe_expert_ffn_i8(s["prob"], api.FFN_ROUTED, s["x_q"], s["x_scale"], s["seg_off"], s["w13"],
                              s["w13_scale"], s["w2"], s["w2_scale"], s["y"], s["ws"])
    return s["y"]


def _quantize(v):
    """Rows to integers (as float32) and scales; the quotient in 64 bits, whose
    nearest integer is that of the real quotient but for ties made by rounding."""
    scale = (v.float().abs().amax(-1) / 127.0).clamp_min(2.0 ** -126)
    return torch.round(v.double() / scale.double()[..., None]).float(), scale


def _int_product(q, w):
    """sum_k q w exactly: 32-bit products of 1024 terms stay below 2^24."""
    acc = None
    for k in range(0, q.shape[-1], 1024):
        part = (q[:, k:k + 1024] @ w[:, k:k + 1024].float().t()).to(torch.int32)
        acc = part if acc is None else acc.add_(part)
    return acc


def _scaled(acc, row_scale, col_scale):
    return acc.double() * (row_scale.double()[:, None] * col_scale.double()[None, :])


def _plain_linear(s):
    q, scale = _quantize(s["x"])
    off = s["seg_off"].tolist()
    y = torch.zeros((q.shape[0], s["w"].shape[1]), dtype=s["x"].dtype, device="cuda")
    for g in range(len(off) - 1):
        a, b = off[g], off[g + 1]
        if b > a:
            y[a:b] = _scaled(_int_product(q[a:b], s["w"][g]), scale[a:b], s["w_scale"][g]).to(y.dtype)
    return y


def _i8_expert(q, scale, w13, w13_scale, w2, w2_scale):
    """One SwiGLU expert on quantised rows, 64-bit values (the hidden row is
    rounded to integers, so values next to a border matter)."""
    F = w13.shape[0] // 2
    gate = _scaled(_int_product(q, w13[:F]), scale, w13_scale[:F])
    h = gate * torch.sigmoid(gate) * _scaled(_int_product(q, w13[F:]), scale, w13_scale[F:])
    hs = (h.abs().amax(-1) / 127.0).float().clamp_min(2.0 ** -126)
    hq = torch.round(h / hs.double()[:, None]).float()
    return _scaled(_int_product(hq, w2), hs, w2_scale)


def _plain_ffn(s):
    q, scale = _quantize(s["x"])
    off = s["seg_off"].tolist()
    y = torch.zeros_like(s["x"])
    for g in range(len(off) - 1):
        a, b = off[g], off[g + 1]
        if b > a:
            y[a:b] = _i8_expert(q[a:b], scale[a:b], s["w13"][g], s["w13_scale"][g], s["w2"][g],
                                s["w2_scale"][g]).to(y.dtype)
    return y


def _expert(x, w13, w2):
    F = w13.shape[0] // 2
    gate = x @ w13[:F].float().t()
    return (gate * torch.sigmoid(gate) * (x @ w13[F:].float().t())) @ w2.float().t()


def _plain_few(s):
    c = s["case"]
    T, E, K, F, Ns = c["T"], c["E"], c["K"], c["F"], c["Ns"]
    i8 = c["weights"] == "i8"
    # router: the choice of experts is decided next to a border, so in 64 bits
    logits = s["x"].double() @ s["w_gate"].double().t()
    if s["logit_offset"] is not None:
        logits = logits + s["logit_offset"].double()
    logits = logits.float()
    e = torch.exp(logits.double() - logits.double().amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    score = logits.double() if s["sel_bias"] is None else p + s["sel_bias"].double()
    idx = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :K]
    w = torch.gather(e, 1, idx)
    w = (w / w.sum(-1, keepdim=True)).float()
    # capacity: earlier tokens first
    chosen = torch.zeros((T, E), dtype=torch.int32, device="cuda").scatter_(1, idx, 1)
    counts = chosen.sum(0)
    rank = torch.gather(chosen.cumsum(0) - chosen, 1, idx)
    cap = T if c["C"] <= 0 else min(T, math.ceil(c["C"] * (T * K) / E))
    kept = counts.clamp(max=cap)
    seg = kept.cumsum(0) - kept
    slot = torch.where(rank < cap, seg[idx] + rank, -1)
    f = counts.double() / (T * K)
    P = p.mean(0)
    stats = torch.cat([f, P, (ALPHA * E * (f * P).sum())[None]]).float()
    # experts
    y = torch.zeros((T, c["d"]), dtype=torch.float64 if i8 else torch.float32, device="cuda")
    q, scale = _quantize(s["x"]) if i8 else (s["x"].float(), None)
    if Ns and i8:  # the shared experts are one wide expert: a scale per token and channel over all of them
        wide13 = torch.cat([s["w13_shared"][:, :F].reshape(Ns * F, -1), s["w13_shared"][:, F:].reshape(Ns * F, -1)])
        wide_s = torch.cat([s["w13_shared_scale"][:, :F].reshape(-1), s["w13_shared_scale"][:, F:].reshape(-1)])
        y += _i8_expert(q, scale, wide13, wide_s, s["w2_shared"].permute(1, 0, 2).reshape(c["d"], -1),
                        s["w2_shared_scale"])
    elif Ns:
        for n in range(Ns):
            y += _expert(q, s["w13_shared"][n], s["w2_shared"][n])
    for ex in torch.nonzero(counts).flatten().tolist():
        tok, k = torch.nonzero((idx == ex) & (slot >= 0), as_tuple=True)
        if i8:
            out = _i8_expert(q[tok], scale[tok], s["w13"][ex], s["w13_scale"][ex], s["w2"][ex], s["w2_scale"][ex])
        else:
            out = _expert(q[tok], s["w13"][ex], s["w2"][ex])
        y.index_add_(0, tok, w[tok, k].to(y.dtype)[:, None] * out)
    return dict(y=y.to(s["x"].dtype), logits=logits, topk_idx=idx.int(), topk_w=w, counts=counts.int(),
                slot_of=slot.int(), stats=stats)


# ------------------------------------------------------------------ the least a pass has to do
def _few_load(case):
    """Routed experts with rows, and kept rows, averaged over a few draws of
    the case's own routing distribution."""
    T, E, K = case["T"], case["E"], case["K"]
    cap = T if case["C"] <= 0 else min(T, math.ceil(case["C"] * (T * K) / E))
    g = torch.Generator().manual_seed(1)
    live = kept = 0.0
    for _ in range(16):
        l = torch.randn((T, E), generator=g)
        if case["zipf"] > 0:
            l = l - case["zipf"] * torch.log((torch.randperm(E, generator=g) + 1).float())
        if case["bias"] > 0:
            l = torch.softmax(l, -1) + (torch.rand(E, generator=g) * 2 - 1) * case["bias"]
        n = torch.bincount(torch.topk(l, K, -1).indices.flatten(), minlength=E)
        live += float((n > 0).sum()) / 16
        kept += float(n.clamp(max=cap).sum()) / 16
    return live, kept


def work(case):
    if case["op"] == "linear":
        rows, G, K, N = case["rows"], case["G"], case["K"], case["N"]
        es = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=rows * K * es + min(G, rows) * N * (K + 4) + rows * N * es, flops=2 * rows * K * N)
    if case["op"] == "ffn":
        rows, G, d, F = case["rows"], case["G"], case["d"], case["F"]
        return dict(bytes=4 * rows * d + min(G, rows) * (3 * F * d + 4 * (2 * F + d)), flops=6 * rows * d * F)
    T, d, E, K, F, Ns = (case[k] for k in ("T", "d", "E", "K", "F", "Ns"))
    live, kept = _few_load(case)
    es = 2 if case["dtype"] == "bf16" else 4
    ws = 1 if case["weights"] == "i8" else es
    per_expert = 3 * F * d * ws + (4 * (2 * F + d) if case["weights"] == "i8" else 0)
    return dict(bytes=int((live + Ns) * per_expert + E * d * es + 2 * T * d * es + 4 * T * E + 12 * T * K + 12 * E),
                flops=int(6 * d * F * (kept + Ns * T) + 2 * T * E * d + 2 * kept * d))


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_quantize(v):
    v = v.to(torch.float64)
    scale = torch.clamp((torch.amax(torch.abs(v), dim=1) / 127).to(torch.float32), min=2.0 ** -126)
    scale = scale.to(torch.float64)
    return torch.round(v / scale.unsqueeze(1)), scale


def _exact_i8_ffn(q, scale, wg, sg, wu, su, w2, s2):
    """SwiGLU on integer rows, everything in float64 (integers up to 2^53 are exact there)."""
    g = torch.matmul(q, wg.double().T) * scale.unsqueeze(1) * sg.double()
    u = torch.matmul(q, wu.double().T) * scale.unsqueeze(1) * su.double()
    hq, hs = _exact_quantize(g / (1 + torch.exp(-g)) * u)
    return torch.matmul(hq, w2.double().T) * hs.unsqueeze(1) * s2.double()


def _exact_linear(case, s):
    out = torch.zeros((case["rows"], case["N"]), dtype=torch.float64, device="cuda")
    off = s["seg_off"].cpu().numpy()
    for g in range(case["G"]):
        rows = slice(int(off[g]), int(off[g + 1]))
        q, scale = _exact_quantize(s["x"][rows]) if off[g + 1] > off[g] else (None, None)
        if q is not None:
            out[rows] = torch.matmul(q, s["w"][g].double().T) * scale.unsqueeze(1) * s["w_scale"][g].double()
    return out


def _exact_ffn(case, s):
    F = case["F"]
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    off = s["seg_off"].cpu().numpy()
    for g in range(case["G"]):
        rows = slice(int(off[g]), int(off[g + 1]))
        if off[g + 1] > off[g]:
            q, scale = _exact_quantize(s["x"][rows])
            out[rows] = _exact_i8_ffn(q, scale, s["w13"][g, :F], s["w13_scale"][g, :F], s["w13"][g, F:],
                                      s["w13_scale"][g, F:], s["w2"][g], s["w2_scale"][g])
    return out


def _exact_few(case, s):
    T, E, K, F, Ns, d = (case[k] for k in ("T", "E", "K", "F", "Ns", "d"))
    i8 = case["weights"] == "i8"
    x = s["x"].double()
    logits = torch.einsum("td,ed->te", x, s["w_gate"].double())
    if s["logit_offset"] is not None:
        logits = logits + s["logit_offset"].double()
    p = torch.softmax(logits, dim=1)
    # token by token on the host: best score first, then the lower index; earlier tokens take an expert's places
    l32 = logits.float().double().cpu().tolist()
    score = l32 if s["sel_bias"] is None else (p + s["sel_bias"].double()).cpu().tolist()
    limit = None if case["C"] <= 0 else math.ceil(case["C"] * (T * K) / E)
    taken, chosen = [0] * E, []
    for t in range(T):
        best = sorted(range(E), key=lambda e: (-score[t][e], e))[:K]
        ranks = [taken[e] for e in best]
        for e in best:
            taken[e] += 1
        chosen.append((best, ranks))
    first, total = [], 0
    for e in range(E):
        first.append(total)
        total += taken[e] if limit is None else min(taken[e], limit)
    weight = [[math.exp(l32[t][e] - max(l32[t])) for e in chosen[t][0]] for t in range(T)]
    weight = [[v / math.fsum(row) for v in row] for row in weight]
    slots = [[first[e] + r if limit is None or r < limit else -1 for e, r in zip(*chosen[t])] for t in range(T)]

    def through(rows, w13, w2, w13_scale, w2_scale, q):
        if i8:
            half = w13.shape[0] // 2
            return _exact_i8_ffn(q[0][rows], q[1][rows], w13[:half], w13_scale[:half], w13[half:], w13_scale[half:],
                                 w2, w2_scale)
        half = w13.shape[0] // 2
        g, u = x[rows] @ w13[:half].double().T, x[rows] @ w13[half:].double().T
        return (g / (1 + torch.exp(-g)) * u) @ w2.double().T

    q = _exact_quantize(s["x"]) if i8 else None
    y = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    every = list(range(T))
    if Ns and i8:  # one expert of width Ns F
        order = [n * 2 * F + f for n in range(Ns) for f in range(F)]
        order += [n * 2 * F + F + f for n in range(Ns) for f in range(F)]
        order = torch.tensor(order, device="cuda")
        y += through(every, s["w13_shared"].reshape(-1, d)[order],
                     torch.cat([s["w2_shared"][n] for n in range(Ns)], dim=1),
                     s["w13_shared_scale"].reshape(-1)[order], s["w2_shared_scale"], q)
    for n in range(0 if i8 else Ns):
        y += through(every, s["w13_shared"][n], s["w2_shared"][n], None, None, None)
    for e in range(E):
        hits = [(t, k) for t in range(T) for k in range(K) if chosen[t][0][k] == e and slots[t][k] >= 0]
        if hits:
            out = through([t for t, _ in hits], s["w13"][e], s["w2"][e], s["w13_scale"][e] if i8 else None,
                          s["w2_scale"][e] if i8 else None, q)
            for row, (t, k) in enumerate(hits):
                y[t] += weight[t][k] * out[row]

    def dev(v, dt):
        return torch.tensor(v, dtype=dt, device="cuda")

    f = dev(taken, torch.float64) / (T * K)
    stats = torch.cat([f, p.mean(dim=0), (ALPHA * E * torch.sum(f * p.mean(dim=0))).reshape(1)])
    return dict(y=y, logits=logits, topk_idx=dev([c[0] for c in chosen], torch.int32),
                topk_w=dev(weight, torch.float64), counts=dev(taken, torch.int32), slot_of=dev(slots, torch.int32),
                stats=stats)


def exact(case, seed):
    return {"few": _exact_few, "ffn": _exact_ffn, "linear": _exact_linear}[case["op"]](case, _inputs(case, seed))
