"""Plain 64-bit forms of the few-token layer and of the 8-bit products, and the
error bounds their tests use.  Torch float64 on the CPU, loops over tokens and
experts; nothing of the library is used.

Error counting (u = 2^-24): a 32-bit sum of n products is off by at most
(n + 2) u times the sum of the magnitudes; a rounding to BF16 by 2^-8 of the
value; silu(g) u computed in FP32 from exact g, u by 2^-19 relative for |g| <= 40
(expf's argument g log2(e) rounded: 40 * 2^-24 * 1.45, under 2^-18.1 absolute in the
exponent, i.e. under 2^-18.6 relative in exp, whose weight in the quotient is at
most 1; two divisions / products more: together under 2^-18)."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
BF16_HALF = 2.0 ** -8
SILU = 2.0 ** -18


def quantize(x: torch.Tensor):
    """(q float64 integers, scale float64) of rows: s = max(fl32(max|v| *
    fl32(1 / 127)), 2^-126), q the nearest integer to v / s, ties to even;
    non-finite rows NaN, 0."""
    x = x.double()
    amax = x.abs().amax(-1).float()
    s = (amax * torch.tensor(1.0 / 127.0, dtype=torch.float32)).clamp(min=2.0 ** -126).double()
    q = torch.round(x / s[..., None])
    bad = ~torch.isfinite(x).all(-1)
    s[bad] = math.nan
    q[bad] = 0.0
    return q, s


def silu_mul(g, u):
    return g * torch.sigmoid(g) * u


def ffn_i8(q, s, w13, s13, w2, s2):
    """y and the bound on an FP32 evaluation of it (before the last rounding):
    a hidden value within its own error of a tie may round either way, one step
    of hs times the weight.  q float64 integers, w int8."""
    F = w13.shape[0] // 2
    z = (q @ w13.double().T) * (s[:, None] * s13.double())
    h = silu_mul(z[:, :F], z[:, F:])
    hq, hs = quantize(h)
    v = h / hs[:, None]
    # g and u: 3 roundings each; then silu; hs itself: its maximum's error and 1 rounding
    rel = 8 * U + 2 * SILU
    near = ((v - torch.floor(v) - 0.5).abs() <= v.abs() * rel + 1e-30).double()
    w = w2.double()
    y = (hq @ w.T) * (hs[:, None] * s2.double())
    flips = (near @ w.abs().T) * (hs[:, None] * s2.double().abs())
    return y, flips + (SILU + 8 * U) * y.abs()


def route(logits, K, bias=None, bias_on_logit=False):
    """idx, w, p from float64 logits (already rounded to float32 where the
    library rounds them); ties to the lower index."""
    l = logits.double()
    p = torch.softmax(l, -1)
    score = l if bias is None else (l + bias.double() if bias_on_logit else p + bias.double())
    idx = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :K]
    g = torch.gather(l, 1, idx)
    return idx, torch.softmax(g, -1), p


def dispatch(idx, E, caps):
    """counts, kept, seg_off, slot_of; caps [E] (negative: no limit)."""
    T, K = idx.shape
    counts = [0] * E
    rank = [[0] * K for _ in range(T)]
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k])
            rank[t][k] = counts[e]
            counts[e] += 1
    kept = [c if caps[e] < 0 else min(c, caps[e]) for e, c in enumerate(counts)]
    off = [0]
    for k in kept:
        off.append(off[-1] + k)
    slot = [[off[int(idx[t, k])] + rank[t][k] if rank[t][k] < kept[int(idx[t, k])] else -1 for k in range(K)]
            for t in range(T)]
    return (torch.tensor(counts, dtype=torch.int32), torch.tensor(kept, dtype=torch.int32),
            torch.tensor(off, dtype=torch.int32), torch.tensor(slot, dtype=torch.int32))


def expert(x, w13, w2, bf16):
    """One SwiGLU expert on float64 rows and the bound on the library's form:
    32-bit sums, the hidden row kept in FP32 (False), rounded to BF16 (True), or
    kept as a sum of two BF16 ("pair")."""
    F, d = w13.shape[0] // 2, w13.shape[1]
    w13, w2 = w13.double(), w2.double()
    z, za = x @ w13.T, (x.abs() @ w13.abs().T) * ((d + 2) * U)
    g, u = z[:, :F], z[:, F:]
    h = silu_mul(g, u)
    # |d silu / dg| <= 1.1; the error of g times |u|, of u times |silu(g)|
    eh = 1.1 * za[:, :F] * (u.abs() + za[:, F:]) + (g * torch.sigmoid(g)).abs() * za[:, F:] + SILU * h.abs()
    if bf16:
        # a pair: the rest, at most 2^-8 of h, is off by 2^-8 of itself; the product with each part sums F terms
        eh = eh + BF16_HALF ** (2 if bf16 == "pair" else 1) * (h.abs() + eh)
    y = h @ w2.T
    ey = eh @ w2.abs().T + ((h.abs() + eh) @ w2.abs().T) * ((F + 8) * U * (2 if bf16 == "pair" else 1))
    return y, ey


def few_layer(inp: dict, K: int, caps, bf16, bias_on_logit=False, logits=None):
    """The layer from CPU inputs: dict of routing, y and its bound (before the
    rounding to the activations' type), and mag, the magnitudes of the expert
    outputs that make up y (times their gates): a form that rounds them to BF16
    first is off by 2^-8 mag more."""
    x = inp["x"].double()
    T, d = x.shape
    E = inp["w13"].shape[0]
    i8 = inp["w13"].dtype == torch.int8
    if logits is None:
        logits = x @ inp["w_gate"].double().T
        if inp.get("logit_offset") is not None:
            logits = logits + torch.as_tensor(inp["logit_offset"]).double()
        logits = logits.float().double()
    bias = inp.get("sel_bias")
    idx, w, p = route(logits, K, None if bias is None else torch.as_tensor(bias), bias_on_logit)
    counts, kept, off, slot = dispatch(idx, E, caps)
    y = torch.zeros((T, d), dtype=torch.float64)
    ey, mag = torch.zeros_like(y), torch.zeros_like(y)
    if i8:
        q, s = quantize(inp["x"])
    if inp.get("w13_shared") is not None:
        Ns, F2, _ = inp["w13_shared"].shape
        F = F2 // 2
        if i8:  # one expert of width N_s F
            w13 = torch.cat([inp["w13_shared"][:, :F].reshape(Ns * F, d), inp["w13_shared"][:, F:].reshape(Ns * F, d)])
            s13 = torch.cat([inp["w13_shared_scale"][:, :F].reshape(-1), inp["w13_shared_scale"][:, F:].reshape(-1)])
            a, b = ffn_i8(q, s, w13, s13, inp["w2_shared"].permute(1, 0, 2).reshape(d, Ns * F), inp["w2_shared_scale"])
            y, ey, mag = y + a, ey + b, mag + a.abs()
        else:
            for n in range(Ns):
                a, b = expert(x, inp["w13_shared"][n], inp["w2_shared"][n], bf16)
                y, ey, mag = y + a, ey + b, mag + a.abs()
    for e in range(E):
        tok, k = torch.nonzero((idx == e) & (slot >= 0), as_tuple=True)
        if len(tok) == 0:
            continue
        if i8:
            a, b = ffn_i8(q[tok], s[tok], inp["w13"][e], inp["w13_scale"][e], inp["w2"][e], inp["w2_scale"][e])
        else:
            a, b = expert(x[tok], inp["w13"][e], inp["w2"][e], bf16)
        y[tok] += w[tok, k][:, None] * a
        ey[tok] += w[tok, k][:, None] * (b + 8 * U * a.abs())
        mag[tok] += w[tok, k][:, None] * a.abs()
    ey = ey + (K + 8) * U * y.abs()
    return dict(logits=logits, topk_idx=idx.int(), topk_w=w, p=p, counts=counts, kept=kept, seg_off=off, slot_of=slot,
                y=y, bound=ey, mag=mag)
