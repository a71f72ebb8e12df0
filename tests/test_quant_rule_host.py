"""The scale of an 8-bit row, fl32(max|v| * fl32(1/127)), against the correctly
rounded quotient max|v| / 127: how far the two rules are apart, and that a row
rounded by either is off by half a step (CPU, 64-bit forms)."""
import torch

import serving_ref as ref

INV = torch.tensor(1.0 / 127.0, dtype=torch.float32)


def ulps(a, b):
    return (a.view(torch.int32) - b.view(torch.int32)).abs()


def test_the_two_scales_are_at_most_one_bit_apart():
    """Every FP32 significand (the exponent only shifts both)."""
    m = (torch.arange(1 << 23, dtype=torch.int32) + (127 << 23)).view(torch.float32)
    product, quotient = m * INV, (m.double() / 127).float()
    assert int(ulps(product, quotient).max()) == 1
    share = float((product != quotient).double().mean())
    assert 1 / 22 < share < 1 / 21
    bf16 = (1 + torch.arange(128) / 128).float()     # 6 of the 128 BF16 significands
    assert int((bf16 * INV != (bf16.double() / 127).float()).sum()) == 6


def rows_of_every_bf16_maximum():
    """Row i: maximum 1 + i / 128, its half (a tie or next to one), and the BF16
    values around every other tie."""
    m = 1 + torch.arange(128).double() / 128
    ties = (torch.arange(-63, 64).double() + 0.5)[None] * m[:, None] / 127
    x = torch.cat([m[:, None], m[:, None] / 2, -m[:, None] / 2, ties], 1).bfloat16()
    up, down = (x.view(torch.int16) + 1).view(torch.bfloat16), (x.view(torch.int16) - 1).view(torch.bfloat16)
    x = torch.cat([x, up[:, 1:], down[:, 1:]], 1)
    return torch.cat([x, torch.zeros((128, -x.shape[1] % 16), dtype=torch.bfloat16)], 1)


def test_rows_rounded_by_either_rule_are_off_by_half_a_step():
    x = rows_of_every_bf16_maximum()
    q, s = ref.quantize(x)
    assert torch.equal(s.float(), x.float().amax(1) * INV)
    s2 = (x.double().abs().amax(1) / 127).float().double()
    q2 = torch.round(x.double() / s2[:, None])
    moved = q != q2
    assert int(moved.sum()) > 0 and float((q - q2).abs().max()) == 1.0
    assert not moved[s == s2].any()                  # only where the scales differ, and only next to ties
    v = x.double() / s[:, None]
    assert float(((v - torch.floor(v) - 0.5).abs() / v.abs())[moved].max()) <= 2.0 ** -23
    for a, b in ((q, s), (q2, s2)):
        # the maximum itself may lie 127 (1 + 2^-23) steps out
        assert float(((x.double() - a * b[:, None]).abs() / b[:, None]).max()) <= 0.5 + 127 * 2.0 ** -23
        assert float(a.abs().max()) == 127.0
