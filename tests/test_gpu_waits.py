"""Waits that run out in the products by expert and in the 4-bit products.

A wait is made to run out by moe_debug_never_signal (every block with work waits for a signal
that is never given) or by a limit of 1 ns.  The call then reports it; with the hooks off the
next call, launched right behind it, gives its usual bits: no copy of the call that gave up
may still be on its way into the shared memory that the next call's blocks get.
"""

import pytest
import torch

import sparse_moe_layer_02_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
TIMEOUT = -6


@pytest.fixture(autouse=True)
def _hooks_off():
    yield
    moe.moe_debug_never_signal(False)
    moe.moe_debug_set_wait_limit_ns(0)


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(BF16)


def _grouped(sizes, M, K):
    g = torch.Generator(device=DEV).manual_seed(1)
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    x, W, dy = _randn(g, sum(sizes), K), _randn(g, len(sizes), M, K), _randn(g, sum(sizes), M)
    return [lambda: moe.moe_grouped_linear(x, W, off), lambda: moe.moe_grouped_linear_dgrad(dy, W, off),
            lambda: moe.moe_grouped_linear_wgrad(dy, x, off)]


def _linear(N, M, K, G):
    g = torch.Generator(device=DEV).manual_seed(2)
    q, s = moe.moe_quantize(_randn(g, M, K, std=0.02), G)
    x = _randn(g, N, K)
    return [lambda: moe.moe_linear_quant(x, q, s)]


def _layer(N, D, E, k, d, G):
    g = torch.Generator(device=DEV).manual_seed(3)
    pair = lambda *shape: moe.moe_quantize(_randn(g, *shape, std=0.05), G)
    w = pair(E, 2 * d, D), pair(E, D, d), pair(2 * d, D), pair(D, d)
    x = _randn(g, N, D)
    ids = torch.rand((N, E), generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
    tw = torch.rand((N, k), generator=g, device=DEV)
    return [lambda: moe.moe_forward_quant(x, *w, ids, tw)]


CASES = {
    "grouped": lambda: _grouped([700, 0, 300], 1024, 2048),       # a tile a block
    "grouped_shared": lambda: _grouped([2000, 40], 128, 2048),    # a cluster's blocks share a tile
    "grouped_many": lambda: _grouped([600] * 24, 1024, 128),      # tiles of two stages, several a block
    "linear_1": lambda: _linear(1, 1024, 4096, 64),
    "linear_16": lambda: _linear(16, 40000, 256, 32),             # short sums, more tiles than places
    "linear_20": lambda: _linear(20, 1024, 4096, 64),
    "linear_40": lambda: _linear(40, 1024, 4096, 64),             # shared by clusters
    "linear_97": lambda: _linear(97, 20480, 256, 32),             # two stages a tile
    "layer_1": lambda: _layer(1, 512, 6, 2, 512, 64),
    "layer_5": lambda: _layer(5, 512, 6, 2, 512, 64),
    "layer_20": lambda: _layer(20, 512, 6, 2, 512, 32),
    "layer_97": lambda: _layer(97, 1024, 24, 4, 1024, 128),
}


@pytest.mark.parametrize("name", list(CASES))
def test_a_signal_that_never_comes_is_reported(name):
    calls = CASES[name]()
    want = [f() for f in calls]
    assert moe.moe_device_status() == 0
    for limit in (2_000_000, 1):
        for f, w in zip(calls, want):
            for _ in range(4):
                moe.moe_debug_set_wait_limit_ns(limit)
                moe.moe_debug_never_signal(True)
                f()
                moe.moe_debug_never_signal(False)
                moe.moe_debug_set_wait_limit_ns(0)
                got = f()
                assert moe.moe_device_status() == TIMEOUT
                assert torch.equal(got, w)
                assert moe.moe_device_status() == 0


@pytest.mark.parametrize("name", list(CASES))
def test_a_call_that_reports_nothing_is_right(name):
    """With a limit of 1 ns a call's waits may run out or not; without a report its results hold."""
    calls = CASES[name]()
    want = [f() for f in calls]
    assert moe.moe_device_status() == 0
    for f, w in zip(calls, want):
        for _ in range(8):
            moe.moe_debug_set_wait_limit_ns(1)
            got = f()
            moe.moe_debug_set_wait_limit_ns(0)
            status = moe.moe_device_status()
            assert status in (0, TIMEOUT)
            if status == 0:
                assert torch.equal(got, w)
            assert torch.equal(f(), w)
    assert moe.moe_device_status() == 0
