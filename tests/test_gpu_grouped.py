"""Products grouped by expert against fp64 (moe_grouped_linear and its gradients).

Tolerances.  A bf16 output is one rounding (half a step, 2^-8 relative) of an fp32 sum
of exact products.  The tensor core's sum is taken to lose at most one step of 2^-22 of
the largest partial sum per 16 products, so over n products at most n/16 * 2^-22 of
S = sum |a b|.  An fp32 output is a chain of n fused multiply-adds: at most n * 2^-24 * S.
Each element is held to that bound of its own S.
"""

import numpy as np
import pytest
import torch

import sparse_moe_layer_02_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _case(sizes, M, K, dtype, lead=0, spare=0, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    E, rows = len(sizes), lead + sum(sizes) + spare
    off = torch.tensor([lead] + (lead + np.cumsum(sizes)).tolist(), dtype=torch.int32, device=DEV)
    mk = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)
    return mk(rows, K), mk(E, M, K), mk(rows, M), off


def _check(got, exact, mass, n, dtype):
    exact, mass = exact.double(), mass.double()
    if dtype == BF16:
        tol = exact.abs() * 2.0 ** -8 + mass * (n / 16 + 1) * 2.0 ** -22 * (1 + 2.0 ** -8)
    else:
        tol = mass * (n + 1) * 2.0 ** -24
    bad = ~((got.double() - exact).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                           got[bad][:4].tolist(), exact[bad][:4].tolist())


def _oracle(x, W, dy, off):
    o = off.tolist()
    y, ym = (torch.zeros(dy.shape, device=DEV, dtype=torch.float64) for _ in range(2))
    dx, dxm = (torch.zeros(x.shape, device=DEV, dtype=torch.float64) for _ in range(2))
    dW, dWm = (torch.zeros(W.shape, device=DEV, dtype=torch.float64) for _ in range(2))
    for e in range(W.shape[0]):
        r = slice(o[e], o[e + 1])
        xe, we, de = x[r].double(), W[e].double(), dy[r].double()
        y[r], ym[r] = xe @ we.t(), xe.abs() @ we.abs().t()
        dx[r], dxm[r] = de @ we, de.abs() @ we.abs()
        dW[e], dWm[e] = de.t() @ xe, de.abs().t() @ xe.abs()
    return (y, ym), (dx, dxm), (dW, dWm)


SHAPES = [
    # sizes, M, K, rows before and behind
    ([1], 8, 8, 0, 0),
    ([3, 0, 5, 1], 64, 72, 0, 0),
    ([128, 256, 64], 256, 128, 0, 0),
    ([127, 129, 0, 0, 1, 31, 33, 63, 65], 264, 200, 0, 7),
    ([0, 0, 17], 136, 520, 5, 300),
    ([300, 16, 15, 48], 1000, 328, 1, 1),
    ([2] * 40 + [0] * 20 + [1] * 9, 520, 1032, 0, 0),
    ([700], 384, 64, 0, 0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes,M,K,lead,spare", SHAPES)
def test_products_match_fp64(sizes, M, K, lead, spare, dtype):
    x, W, dy, off = _case(sizes, M, K, dtype, lead, spare)
    (y, ym), (dx, dxm), (dW, dWm) = _oracle(x, W, dy, off)
    _check(moe.moe_grouped_linear(x, W, off), y, ym, K, dtype)
    _check(moe.moe_grouped_linear_dgrad(dy, W, off), dx, dxm, M, dtype)
    _check(moe.moe_grouped_linear_wgrad(dy, x, off), dW, dWm, max(sizes), dtype)
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("dtype,M,K", [(F32, 4, 12), (F32, 100, 36)])
def test_fp32_rows_of_four(dtype, M, K):
    x, W, dy, off = _case([5, 0, 40], M, K, dtype)
    (y, ym), (dx, dxm), (dW, dWm) = _oracle(x, W, dy, off)
    _check(moe.moe_grouped_linear(x, W, off), y, ym, K, dtype)
    _check(moe.moe_grouped_linear_dgrad(dy, W, off), dx, dxm, M, dtype)
    _check(moe.moe_grouped_linear_wgrad(dy, x, off), dW, dWm, 40, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_no_expert_are_neither_read_nor_written(dtype):
    sizes, lead, spare = [33, 0, 70, 1], 6, 9
    x, W, dy, off = _case(sizes, 136, 80, dtype, lead, spare)
    (y, ym), (dx, dxm), (dW, dWm) = _oracle(x, W, dy, off)
    rest = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    rest[lead:lead + sum(sizes)] = False
    x[rest] = float("nan")
    dy[rest] = float("inf")
    gy = moe.moe_grouped_linear(x, W, off, y=torch.full_like(dy, 7.0))
    gx = moe.moe_grouped_linear_dgrad(dy, W, off, dx=torch.full_like(x, 7.0))
    assert (gy[rest] == 7.0).all() and (gx[rest] == 7.0).all()
    _check(gy[~rest], y[~rest], ym[~rest], 80, dtype)
    _check(gx[~rest], dx[~rest], dxm[~rest], 136, dtype)
    _check(moe.moe_grouped_linear_wgrad(dy, x, off, dW=torch.full_like(W, float("nan"))), dW, dWm,
           max(sizes), dtype)
    assert (moe.moe_grouped_linear(x, W, off)[rest] == 0).all()
    assert (moe.moe_grouped_linear_dgrad(dy, W, off)[rest] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_experts_nan_stays_its_own(dtype):
    """A NaN or infinity in one expert's rows or weights reaches no other expert's results,
    though the tiles of neighbours overlap it."""
    sizes, M, K = [5, 40, 3], 72, 88
    x, W, dy, off = _case(sizes, M, K, dtype)
    (y, ym), (dx, dxm), (dW, dWm) = _oracle(x, W, dy, off)
    x[5:45], dy[5:45], W[1] = float("nan"), float("inf"), float("nan")
    keep = torch.ones(48, dtype=torch.bool, device=DEV)
    keep[5:45] = False
    _check(moe.moe_grouped_linear(x, W, off)[keep], y[keep], ym[keep], K, dtype)
    _check(moe.moe_grouped_linear_dgrad(dy, W, off)[keep], dx[keep], dxm[keep], M, dtype)
    got = moe.moe_grouped_linear_wgrad(dy, x, off)
    for e in (0, 2):
        _check(got[e], dW[e], dWm[e], 5, dtype)
    assert torch.isnan(got[1]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_rows(dtype):
    x, W, dy, off = _case([0, 0], 16, 24, dtype)
    assert moe.moe_grouped_linear(x, W, off).shape == (0, 16)
    assert moe.moe_grouped_linear_dgrad(dy, W, off).shape == (0, 24)
    assert (moe.moe_grouped_linear_wgrad(dy, x, off, dW=torch.ones_like(W)) == 0).all()
    x, W, dy, off = _case([0, 0], 16, 24, dtype, spare=3)  # rows, but none of any expert
    assert (moe.moe_grouped_linear(x, W, off) == 0).all()
    assert (moe.moe_grouped_linear_wgrad(dy, x, off) == 0).all()
    assert moe.moe_device_status() == 0


def test_offsets_out_of_order_are_made_safe_and_reported():
    x, W, dy, _ = _case([20, 20], 16, 24, BF16)
    off = torch.tensor([-3, 900, 10], dtype=torch.int32, device=DEV)
    safe = torch.tensor([0, 40, 40], dtype=torch.int32, device=DEV)
    got = moe.moe_grouped_linear(x, W, off)
    assert moe.moe_device_status() == -7
    assert torch.equal(got, moe.moe_grouped_linear(x, W, safe))
    got = moe.moe_grouped_linear_wgrad(dy, x, off)
    assert moe.moe_device_status() == -7
    assert torch.equal(got, moe.moe_grouped_linear_wgrad(dy, x, safe))
    assert moe.moe_device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_by_autograd(dtype):
    x, W, dy, off = _case([9, 0, 30], 64, 48, dtype, spare=4)
    (_, _), (dx, dxm), (dW, dWm) = _oracle(x, W, dy, off)
    x.requires_grad_(True)
    W.requires_grad_(True)
    y = moe.moe_grouped_linear(x, W, off)
    y.backward(dy)
    _check(x.grad, dx, dxm, 64, dtype)
    _check(W.grad, dW, dWm, 30, dtype)
    only, = torch.autograd.grad(moe.moe_grouped_linear(x, W, off).sum(), [W])  # expanded dy
    ones = torch.ones_like(dy)
    assert torch.equal(only, moe.moe_grouped_linear_wgrad(ones, x.detach(), off))


def test_gradient_against_differences():
    """fp32 against central differences of the fp64 formula."""
    x, W, dy, off = _case([4, 0, 3], 8, 12, F32, seed=3)
    o = off.tolist()

    def loss(xv, Wv):
        return sum(((xv[o[e]:o[e + 1]] @ Wv[e].t()) * dy[o[e]:o[e + 1]].double()).sum()
                   for e in range(3))
    x64, W64, h = x.double(), W.double(), 1e-4
    gx = moe.moe_grouped_linear_dgrad(dy, W, off)
    gW = moe.moe_grouped_linear_wgrad(dy, x, off)
    for g, v, at in ((gx, x64, (2, 5)), (gx, x64, (6, 11)), (gW, W64, (0, 7, 3)), (gW, W64, (2, 0, 0))):
        keep = v[at].item()
        v[at] = keep + h
        hi = loss(x64, W64)
        v[at] = keep - h
        lo = loss(x64, W64)
        v[at] = keep
        # the loss is linear in each entry: only roundings are left (sums below 100)
        assert abs(((hi - lo) / (2 * h)).item() - g[at].item()) <= 1e-4


def test_other_stream_and_graph():
    x, W, dy, off = _case([50, 3, 130], 264, 136, BF16)
    want = [moe.moe_grouped_linear(x, W, off), moe.moe_grouped_linear_dgrad(dy, W, off),
            moe.moe_grouped_linear_wgrad(dy, x, off)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, dx, dW = (torch.empty_like(t) for t in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_grouped_linear(x, W, off, y=y)
        moe.moe_grouped_linear_dgrad(dy, W, off, dx=dx)
        moe.moe_grouped_linear_wgrad(dy, x, off, dW=dW)
    for _ in range(2):
        for t in (y, dx, dW):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dW), want))
    # new segments in the same buffers, without a new capture
    off.copy_(torch.tensor([0, 100, 100, 183], dtype=torch.int32, device=DEV))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, moe.moe_grouped_linear(x, W, off))
    assert torch.equal(dW, moe.moe_grouped_linear_wgrad(dy, x, off))
    assert moe.moe_device_status() == 0


def test_refusals():
    x, W, dy, off = _case([5, 6], 16, 24, BF16)
    for bad in (lambda: moe.moe_grouped_linear(x[:, :16], W, off),
                lambda: moe.moe_grouped_linear(x.t().contiguous().t(), W, off),
                lambda: moe.moe_grouped_linear(x, W.float(), off),
                lambda: moe.moe_grouped_linear(x, W, off.long()),
                lambda: moe.moe_grouped_linear(x, W, off[:2]),
                lambda: moe.moe_grouped_linear(x, W.cpu(), off),
                lambda: moe.moe_grouped_linear(x, W, off, y=torch.empty_like(x)),
                lambda: moe.moe_grouped_linear_dgrad(x, W, off),
                lambda: moe.moe_grouped_linear_wgrad(dy[:5], x, off)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoEError):  # rows of 16 bytes
        moe.moe_grouped_linear(x[:, :20].contiguous(), W[:, :, :20].contiguous(), off)


def test_capture_over_a_living_eager_pass_is_refused():
    """Autograd would end the process in the captured backward; the captured forward raises."""
    x, W, dy, off = _case([9, 30], 64, 48, BF16)
    x.requires_grad_(True)
    W.requires_grad_(True)
    alive = moe.moe_grouped_linear(x, W, off)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with pytest.raises(ValueError, match="eager"):
        with torch.cuda.graph(g, stream=s):
            moe.moe_grouped_linear(x, W, off)
    torch.cuda.synchronize()
    alive.backward(dy)
    want = x.grad.clone(), W.grad.clone()
    del alive, g
    # with the eager pass gone, forward and backward are captured and replayed
    x.grad = W.grad = None
    with torch.cuda.stream(s):
        for _ in range(2):
            gx, gW = torch.autograd.grad(moe.moe_grouped_linear(x, W, off), [x, W], dy)
    del gx, gW
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gx, gW = torch.autograd.grad(moe.moe_grouped_linear(x, W, off), [x, W], dy)
    for t in (gx, gW):
        t.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(gx, want[0]) and torch.equal(gW, want[1])


def test_an_output_with_gradients_is_refused():
    x, W, dy, off = _case([9, 30], 64, 48, BF16)
    W.requires_grad_(True)
    with pytest.raises(ValueError):
        moe.moe_grouped_linear(x, W, off, y=torch.empty_like(dy))
    with torch.no_grad():
        y = moe.moe_grouped_linear(x, W, off, y=torch.empty_like(dy))
    assert torch.equal(y, moe.moe_grouped_linear(x, W.detach(), off))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_past_32_bits(dtype):
    """More than 2^31 elements of x, and of W: the last rows and the last expert are right.

    fp32 sums are in index order whatever the sizes: equal to those of a small call.  How many
    blocks share a bf16 sum depends on the number of tiles, so those are held to fp64, with
    the bound above and 2 * 2^-22 for the 7 additions of 2^-24 that join 8 shares."""
    def same(got, small, exact, mass, n):
        if dtype == F32:
            assert torch.equal(got, small())
        else:
            _check(got, exact, mass, n + 32, BF16)
    K, M, rows = 4096, 8, 2 ** 31 // 4096 + 700
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    x = torch.zeros((rows, K), dtype=dtype, device=DEV)
    x[-500:] = torch.randn((500, K), generator=g, device=DEV).to(dtype)
    W = torch.randn((2, M, K), generator=g, device=DEV).to(dtype)
    dy = torch.ones((rows, M), dtype=dtype, device=DEV)
    off = torch.tensor([0, rows - 333, rows], dtype=torch.int32, device=DEV)
    xs, small = x[-500:].clone(), torch.tensor([0, 167, 500], dtype=torch.int32, device=DEV)
    (ye, ym), (dxe, dxm), (dWe, dWm) = _oracle(xs, W, dy[-500:], small)
    y = moe.moe_grouped_linear(x, W, off)
    same(y[-500:], lambda: moe.moe_grouped_linear(xs, W, small), ye, ym, K)
    assert (y[:-500] == 0).all()
    del y
    dx = moe.moe_grouped_linear_dgrad(dy, W, off)
    same(dx[-500:], lambda: moe.moe_grouped_linear_dgrad(dy[-500:], W, small), dxe, dxm, M)
    del dx
    dW = moe.moe_grouped_linear_wgrad(dy, x, off)
    same(dW[1], lambda: moe.moe_grouped_linear_wgrad(dy[-500:], xs, small)[1], dWe[1], dWm[1], 333)
    del x, W, dy, dW
    E = 2 ** 31 // (1056 * 4096) + 1  # 497, of at most 512
    W = torch.zeros((E, 1056, 4096), dtype=dtype, device=DEV)
    W[-1] = torch.randn((1056, 4096), generator=g, device=DEV).to(dtype)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[-1] = 500
    one = torch.tensor([0, 500], dtype=torch.int32, device=DEV)
    dy = torch.randn((500, 1056), generator=g, device=DEV).to(dtype)
    (ye, ym), (dxe, dxm), (dWe, dWm) = _oracle(xs, W[-1:], dy, one)
    same(moe.moe_grouped_linear(xs, W, off), lambda: moe.moe_grouped_linear(xs, W[-1:], one), ye, ym, 4096)
    same(moe.moe_grouped_linear_dgrad(dy, W, off), lambda: moe.moe_grouped_linear_dgrad(dy, W[-1:], one), dxe, dxm, 1056)
    dW = moe.moe_grouped_linear_wgrad(dy, xs, off, dW=W)
    same(dW[-1], lambda: moe.moe_grouped_linear_wgrad(dy, xs, one)[0], dWe[0], dWm[0], 500)
    assert (dW[:-1] == 0).all()
    assert moe.moe_device_status() == 0


def test_a_wait_that_runs_out_is_reported_and_leaves_the_device_usable():
    x, W, dy, off = _case([700, 300], 1024, 2048, BF16)
    calls = (lambda: moe.moe_grouped_linear(x, W, off), lambda: moe.moe_grouped_linear_dgrad(dy, W, off),
             lambda: moe.moe_grouped_linear_wgrad(dy, x, off))
    want = [f() for f in calls]
    assert moe.moe_device_status() == 0
    try:
        moe.moe_debug_set_wait_limit_ns(1)
        for f in calls:
            f()
            assert moe.moe_device_status() in (0, -6)
    finally:
        moe.moe_debug_set_wait_limit_ns(0)
    assert all(torch.equal(f(), w) for f, w in zip(calls, want))
    assert moe.moe_device_status() == 0


def test_two_streams_at_once():
    a, b = _case([200, 3, 130], 264, 520, BF16), _case([64] * 9, 512, 256, BF16, seed=1)
    want = [moe.moe_grouped_linear(c[0], c[1], c[3]) for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate((a, b)):
            got[i].append(moe.moe_grouped_linear(c[0], c[1], c[3], stream=streams[i],
                                                 y=torch.empty_like(want[i])))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    assert moe.moe_device_status() == 0


def test_what_a_call_makes_is_memory_of_the_calls_stream():
    # The current stream gives a block back while its last write is still to come; a call on
    # another stream must not be handed that block.
    x, W, dy, off = _case([200, 3, 130], 1288, 2056, BF16)
    other = torch.cuda.Stream()
    for f in (lambda **k: moe.moe_grouped_linear(x, W, off, **k),
              lambda **k: moe.moe_grouped_linear_dgrad(dy, W, off, **k),
              lambda **k: moe.moe_grouped_linear_wgrad(dy, x, off, **k)):
        want = f()
        torch.cuda.synchronize()
        scratch = torch.empty_like(want)
        torch.cuda._sleep(100_000_000)
        scratch.fill_(float("nan"))
        del scratch
        got = f(stream=other)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


# Few tiles with long sums: the k-blocks of a tile are shared by 2, 4 or 8 blocks, whose
# sums are added in fp32 (7 roundings of 2^-24 at most: two more steps of 2^-22, or 32 more
# products to _check).  Shares that differ, experts with no rows or too few for a share.
@pytest.mark.parametrize("sizes,M,K,lead,spare", [
    ([5], 264, 4104, 0, 0), ([130, 0, 3], 2056, 136, 3, 2), ([1700, 0, 2100], 200, 72, 0, 50),
    ([9001], 136, 520, 7, 0), ([40, 2000, 1, 70, 63, 0, 64, 65], 128, 264, 0, 0), ([33], 4096, 2048, 0, 0),
    ([600, 601], 1024, 1536, 0, 0),
    ([3000, 40, 0, 4500, 100], 200, 136, 0, 9)])
def test_products_of_few_tiles_match_fp64(sizes, M, K, lead, spare):
    x, W, dy, off = _case(sizes, M, K, BF16, lead, spare)
    (y, ym), (dx, dxm), (dW, dWm) = _oracle(x, W, dy, off)
    rest = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    rest[lead:lead + sum(sizes)] = False
    x[rest], dy[rest] = float("nan"), float("inf")
    calls = (lambda: moe.moe_grouped_linear(x, W, off), lambda: moe.moe_grouped_linear_dgrad(dy, W, off),
             lambda: moe.moe_grouped_linear_wgrad(dy, x, off))
    for f, t, m, n in zip(calls, (y, dx, dW), (ym, dxm, dWm), (K, M, max(sizes))):
        got = f()
        _check(got, t, m, n + 32, BF16)
        assert all(torch.equal(f(), got) for _ in range(3))
    assert moe.moe_device_status() == 0
    y = moe.moe_grouped_linear(x, W, off, y=torch.full_like(dy, 7.0))
    assert (y[rest] == 7.0).all()


def test_a_wait_that_runs_out_among_few_tiles_leaves_the_device_usable():
    x, W, dy, off = _case([2000, 40], 128, 2048, BF16)
    calls = (lambda: moe.moe_grouped_linear(x, W, off), lambda: moe.moe_grouped_linear_wgrad(dy, x, off))
    want = [f() for f in calls]
    torch.cuda.synchronize()
    moe.moe_debug_set_wait_limit_ns(1)
    try:
        for f in calls:
            f()
            assert moe.moe_device_status() in (0, -6)
    finally:
        moe.moe_debug_set_wait_limit_ns(0)
    assert all(torch.equal(f(), w) for f, w in zip(calls, want))
    assert moe.moe_device_status() == 0
