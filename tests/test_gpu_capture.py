"""Captured training passes of moe_grouped_linear beside living eager ones."""

import pytest
import torch

import sparse_moe_layer_02_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(dtype):
    g = torch.Generator(device=DEV).manual_seed(0)
    mk = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)
    off = torch.tensor([0, 9, 9, 39], dtype=torch.int32, device=DEV)
    return mk(42, 48), mk(3, 64, 48), mk(42, 64), off


@pytest.mark.parametrize("held", ["pass", "node"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_capture_beside_what_a_side_stream_left_alive(dtype, held):
    """A pass warmed up on a side stream stays alive, or a holder of the leaves' accumulation
    nodes made there does (as data-parallel wrappers keep them): a capture on another stream
    joins that stream, and its replays give the eager gradients."""
    x, W, dy, off = _case(dtype)
    x.requires_grad_(True)
    W.requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        if held == "node":
            alive = [torch.autograd.graph.get_gradient_edge(t) for t in (x, W)]
        for _ in range(2):
            want = torch.autograd.grad(moe.moe_grouped_linear(x, W, off), [x, W], dy)
        if held == "pass":
            alive = moe.moe_grouped_linear(x, W, off)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = torch.autograd.grad(moe.moe_grouped_linear(x, W, off), [x, W], dy)
    for t in got:
        t.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x.grad, W.grad = torch.zeros_like(x), torch.zeros_like(W)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        moe.moe_grouped_linear(x, W, off).backward(dy)   # accumulates into the leaves
    for t in (x.grad, W.grad):
        t.zero_()
    g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(x.grad, want[0]) and torch.equal(W.grad, want[1])
    del alive
    assert moe.moe_device_status() == 0


def test_capture_beside_a_pass_of_the_default_stream_is_refused():
    x, W, dy, off = _case(torch.float32)
    W.requires_grad_(True)
    alive = moe.moe_grouped_linear(x, W, off)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError, match="default"):
        with torch.cuda.graph(g):
            moe.moe_grouped_linear(x, W, off)
    torch.cuda.synchronize()
    alive.backward(dy)
    assert torch.equal(W.grad, moe.moe_grouped_linear_wgrad(dy, x, off))
