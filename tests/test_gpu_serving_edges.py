"""Calls of the serving operators that their documents allow and that are easy to
get wrong: first calls on a side stream, forwards in other orders, sizes at the
limits."""
import pytest
import torch

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
