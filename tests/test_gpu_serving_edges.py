"""Calls of the serving operators that their documents allow and that are easy to
get wrong: first calls on a side stream, forwards in other orders, sizes at the
limits."""
import pytest
import torch

from sparse_mixture_experts_04_b200 import api
from test_gpu_few import build, make

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
