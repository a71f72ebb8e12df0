"""The few-token layer when a wait runs out (MOE_B200_TEST_STALL_NS: CTA 0 comes
late to the barriers, the other CTAs give up a quarter of that time before): the
kernel reports MOE_DEV_WAIT_TIMEOUT, takes no row index that nobody wrote (the
workspace and the routing arrays hold values far outside them), and returns; the
next call gives what the one before it gave."""
import time

import pytest
import torch

from sparse_mixture_experts_04_b200 import api
from sparse_mixture_experts_04_b200._lib import DEV_WAIT_TIMEOUT
from test_gpu_few import build, make

pytestmark = pytest.mark.gpu

STALL_NS = "2000000"   # 2 ms instead of the 2 s limit of a real wait


# T <= 8: every CTA ranks all tokens; more: one each, with a grid barrier more
@pytest.mark.parametrize("T,kind", [(4, "bf16"), (40, "bf16"), (3, "f32"), (24, "i8")])
def test_few_layer_wait_timeout_is_reported_and_the_context_stays_usable(T, kind, monkeypatch):
    inp = make(T, 256, 8, 2, 192, 1, kind, 21)
    layer = build(inp, 2, 0.0, api.FLAG_EXTENDED_STATS, None, 1)
    x = inp["x"].cuda()
    good = layer.forward_few(x).clone()
    assert api.read_device_status(layer.few_ws) == 0
    layer.few_ws.fill_(0x7f)
    for k, v in layer.routing.items():
        v.view(torch.int32).fill_(0x7f7f7f7f)
    y = torch.full_like(good, 3.0)
    torch.cuda.synchronize()
    monkeypatch.setenv("MOE_B200_TEST_STALL_NS", STALL_NS)
    t0 = time.monotonic()
    layer.forward_few(x, y)
    bits = api.read_device_status(layer.few_ws)   # synchronises the stream
    assert bits & DEV_WAIT_TIMEOUT, f"status {bits:#x}"
    assert time.monotonic() - t0 < 10.0
    monkeypatch.delenv("MOE_B200_TEST_STALL_NS")
    for _ in range(2):
        assert torch.equal(layer.forward_few(x, y), good)
        assert api.read_device_status(layer.few_ws) == 0
