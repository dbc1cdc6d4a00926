"""Weights in 4 bits with group scales against fp64: conversion, products, whole layer.

Tolerances.  Codes and scales are exact (a quotient of two bf16 values is never within
fp32 rounding of a half without being one).  A product's bf16 output is one rounding (2^-8
relative) of an fp32 sum; codes times tokens are exact, a tensor-core step of 16 products is
taken to lose at most 2^-22 of its largest partial sum, the group scales' multiply-adds and
the sums of slices 2^-24 each, so (K/16 + K/32 + 10) * 2^-22 of S = sum |x w| covers them.
The layer's SwiGLU output h is rounded to bf16 (2^-8 of |h|), after a SwiGLU whose fast
exponential and division are taken at 2^-20; both pass through the down product, where they
weigh |down| |h|.
"""

import numpy as np
import pytest
import torch

import sparse_moe_layer_02_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _codes(q):
    return torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).double() - 8.0


def _values(q, s):
    """fp64 values [.., M, K]."""
    c = _codes(q)
    return c * s.double().transpose(-1, -2).repeat_interleave(c.shape[-1] // s.shape[-2], dim=-1)


def _expected(W, G):
    """Codes (as -8..7) and scales by the definition, in fp64."""
    w = W.double()
    v = w.view(*w.shape[:-1], -1, G)
    top = v.abs().amax(-1)
    s = (top / 7).to(BF16)
    s = torch.where(torch.isfinite(top), s, torch.full_like(s, float("nan")))
    sd = s.double()[..., None]
    c = torch.where(sd > 0, torch.round(v / sd), torch.zeros_like(v)).nan_to_num(0).clamp(-8, 7)
    c = torch.where(torch.isfinite(top)[..., None], c, torch.zeros_like(c))
    return c.view_as(w), s.transpose(-1, -2)


# ------------------------------------------------------------------------- conversion
@pytest.mark.parametrize("lead,M,K,G", [((), 8, 32, 32), ((), 8, 128, 128), ((3,), 40, 192, 64),
                                        ((2, 2), 24, 1408, 128), ((), 264, 352, 32), ((1,), 1000, 320, 64)])
def test_codes_and_scales_are_exact(lead, M, K, G):
    W = _randn(_gen(M + K), *lead, M, K, std=0.02)
    W.view(-1, K)[0, :G] = 0                    # a group of zeros
    W.view(-1, K)[1, :G] *= 2.0 ** -125         # its scale is below bf16's normal numbers
    W.view(-1, K)[2, :G] = 1e-40                # below half of bf16's smallest: scale 0
    q, s = moe.moe_quantize(W, G)
    c, sx = _expected(W, G)
    assert torch.equal(s, sx)
    assert torch.equal(_codes(q), c)
    assert torch.equal(moe.moe_dequantize(q, s), _values(q, s).to(BF16))
    assert torch.isfinite(moe.moe_dequantize(q, s)).all()


def test_halves_round_to_even_and_bad_values_stay_in_their_group():
    W = torch.zeros((16, 64), dtype=BF16, device=DEV)
    W[0, :8] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -7.0])
    W[1, 3], W[1, 40] = float("nan"), 1.0
    W[2, 5], W[3, 33] = float("inf"), -float("inf")
    q, s = moe.moe_quantize(W, 32)
    assert _codes(q)[0, :8].tolist() == [7, 0, 2, 2, 0, -2, -2, -7]
    nan = torch.isnan(s)
    assert nan.nonzero().tolist() == [[0, 1], [0, 2], [1, 3]]
    back = moe.moe_dequantize(q, s)
    bad = nan.t().repeat_interleave(32, dim=1)
    assert torch.isnan(back[bad]).all() and torch.isfinite(back[~bad]).all()
    assert back[1, 40] == _values(q, s)[1, 40].to(BF16)


# ------------------------------------------------------------------------- one matrix
def _product_tol(x, w, K, y):
    mass = x.double().abs() @ w.abs().t()
    return y.abs() * 2.0 ** -8 + mass * (K / 16 + K / 32 + 10) * 2.0 ** -22


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,M,K", [(1, 8, 128), (1, 2816, 4096), (2, 72, 640), (7, 264, 384), (8, 64, 256),
                                   (9, 136, 512), (16, 1000, 896), (17, 128, 1408), (33, 392, 640),
                                   (70, 520, 256), (3, 20000, 128)])
def test_product_matches_fp64(N, M, K, G):
    g = _gen(N * 7 + M + K + G)
    q, s = moe.moe_quantize(_randn(g, M, K, std=0.02), G)
    x = _randn(g, N, K)
    w = _values(q, s)
    y = x.double() @ w.t()
    got = moe.moe_linear_quant(x, q, s)
    assert moe.moe_device_status() == 0
    bad = ~((got.double() - y).abs() <= _product_tol(x, w, K, y))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(),
                           y[bad][:4].tolist())


def test_every_code_in_every_place():
    """One-hot tokens read single weights: every code, row and column lands where it should."""
    M, K, G = 48, 256, 32
    q = torch.arange(M * K // 2, device=DEV, dtype=torch.int64).mul(37).remainder(256).to(torch.uint8)
    q = q.view(M, K // 2)
    s = (torch.arange(K // G * M, device=DEV).remainder(17) + 1).to(BF16).view(K // G, M)
    x = torch.eye(K, dtype=BF16, device=DEV)
    want = _values(q, s).t().to(BF16)          # at most 8 + 5 bits: rounded once
    for n in (1, 8, 16, K):
        for a in range(0, K, n):
            if n < 8 and a > 40:
                break
            assert torch.equal(moe.moe_linear_quant(x[a:a + n], q, s), want[a:a + n]), (n, a)


def test_nan_tokens_and_scales_stay_their_own():
    g = _gen(5)
    q, s = moe.moe_quantize(_randn(g, 104, 384, std=0.02), 64)
    x = _randn(g, 21, 384)
    y = moe.moe_linear_quant(x, q, s)
    x[4], x[20, 383] = float("nan"), float("inf")
    s[5, 100] = float("nan")
    got = moe.moe_linear_quant(x, q, s)
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[4] = keep[20] = False
    keep[:, 100] = False
    assert torch.equal(got[keep], y[keep])
    assert torch.isnan(got[4]).all() and torch.isnan(got[:, 100]).all()
    assert not torch.isfinite(got[20]).any()


# ------------------------------------------------------------------------- whole layer
def _layer(N, D, E, k, d, d_sh, G, seed=0, ids=None):
    g = _gen(seed)
    w = dict(gate_up=moe.moe_quantize(_randn(g, E, 2 * d, D, std=0.05), G),
             down=moe.moe_quantize(_randn(g, E, D, d, std=0.05), G),
             sh_gate_up=moe.moe_quantize(_randn(g, 2 * d_sh, D, std=0.05), G),
             sh_down=moe.moe_quantize(_randn(g, D, d_sh, std=0.05), G))
    x = _randn(g, N, D)
    if ids is None:
        ids = torch.rand((N, E), generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
    tw = torch.rand((N, k), generator=g, device=DEV)
    return x, w, ids, tw


def _swiglu(gu, gate_max, up_max):
    a, u = gu.chunk(2, dim=1)
    a, u = a.clamp(max=gate_max), u.clamp(-up_max, up_max)
    return a * torch.sigmoid(a) * u


def _layer_oracle(x, w, ids, tw, gate_max=float("inf"), up_max=float("inf")):
    """y and the error allowed before its own rounding."""
    xd = x.double()
    E = w["gate_up"][0].shape[0]
    y, tol = torch.zeros_like(xd), torch.zeros_like(xd)
    D = x.shape[1]

    def expert(rows, gu, dn):
        v, m = xd[rows] @ gu.t(), xd[rows].abs() @ gu.abs().t()
        h = _swiglu(v, gate_max, up_max)
        ga, ua = (t.abs() for t in v.chunk(2, dim=1))
        eg, eu = (t * (D / 16 + D / 32 + 10) * 2.0 ** -22 for t in m.chunk(2, dim=1))
        # |d silu| <= 1.1, |silu(a)| <= |a| (or the limit)
        dh = 1.1 * eg * (ua.clamp(max=up_max) + eu) + eu * ga.clamp(max=max(gate_max, 1.0))
        dh = dh + h.abs() * (2.0 ** -8 + 2.0 ** -20) * 1.01
        d = h.shape[1]
        return h @ dn.t(), (dh + h.abs() * (d / 16 + d / 32 + 10) * 2.0 ** -22) @ dn.abs().t()
    o, t = expert(slice(None), _values(*w["sh_gate_up"]), _values(*w["sh_down"]))
    y += o
    tol += t
    for e in range(E):
        rows, slots = (ids == e).nonzero(as_tuple=True)
        if len(rows) == 0:
            continue
        o, t = expert(rows, _values(w["gate_up"][0][e], w["gate_up"][1][e]),
                      _values(w["down"][0][e], w["down"][1][e]))
        c = tw[rows, slots].double()[:, None]
        y.index_add_(0, rows, o * c)
        tol.index_add_(0, rows, t * c + (o * c).abs() * 8 * 2.0 ** -24)
    return y, tol + y.abs() * 2.0 ** -8 * 1.01


def _run(x, w, ids, tw, **kw):
    return moe.moe_forward_quant(x, w["gate_up"], w["down"], w["sh_gate_up"], w["sh_down"], ids, tw, **kw)


@pytest.mark.parametrize("N,D,E,k,d,d_sh,G", [
    (1, 256, 4, 2, 128, 128, 128), (1, 512, 16, 8, 384, 128, 64), (2, 256, 4, 4, 128, 256, 32),
    (5, 384, 8, 1, 256, 128, 128), (8, 256, 3, 3, 96, 160, 32), (13, 256, 40, 8, 128, 128, 64),
    (32, 640, 6, 2, 128, 384, 128), (64, 256, 2, 2, 64, 64, 64), (100, 256, 5, 4, 160, 96, 32),
    (300, 256, 8, 8, 128, 128, 128)])
def test_layer_matches_fp64(N, D, E, k, d, d_sh, G):
    x, w, ids, tw = _layer(N, D, E, k, d, d_sh, G, seed=N + E)
    y, tol = _layer_oracle(x, w, ids, tw)
    got = _run(x, w, ids, tw)
    assert moe.moe_device_status() == 0
    bad = ~((got.double() - y).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), y[bad][:4].tolist())
    assert torch.equal(got, _run(x, w, ids, tw))      # the same bits again


@pytest.mark.parametrize("N", [1, 6, 40])
def test_layer_sentinel_and_the_same_expert_twice(N):
    x, w, ids, tw = _layer(N, 256, 6, 4, 128, 128, 64, seed=2)
    ids[:, 0] = 6                       # no expert
    ids[0, 1:] = 3                      # one expert three times
    if N > 1:
        ids[N - 1] = 6                  # an idle row: the shared expert only
    y, tol = _layer_oracle(x, w, ids, tw)
    got = _run(x, w, ids, tw)
    assert moe.moe_device_status() == 0
    assert ((got.double() - y).abs() <= tol).all()
    ids[0, 0] = 7                       # outside: skipped and reported
    assert torch.equal(_run(x, w, ids, tw), got)
    assert moe.moe_device_status() == -7
    ids[0, 0] = -1
    assert torch.equal(_run(x, w, ids, tw), got)
    assert moe.moe_device_status() == -7


@pytest.mark.parametrize("N", [1, 20])
def test_layer_limits(N):
    x, w, ids, tw = _layer(N, 256, 6, 2, 128, 128, 64, seed=4)
    x *= 4
    y, tol = _layer_oracle(x, w, ids, tw, 1.0, 0.5)
    got = _run(x, w, ids, tw, gate_max=1.0, up_max=0.5)
    assert ((got.double() - y).abs() <= tol).all()
    assert not torch.equal(got, _run(x, w, ids, tw))


def test_layer_agrees_with_the_bf16_layer_on_the_same_weights():
    """Router, 4-bit layer and the bf16 layer on the dequantized weights, as a program runs
    them; the two differ by the rounding of the weights' values and of the partial outputs
    (a few 2^-8 of the output's size)."""
    N, D, E, k, d = 48, 512, 16, 4, 256
    x, w, _, _ = _layer(N, D, E, k, d, d, 128, seed=9)
    g = _gen(1)
    idx, tw = moe.moe_router(x, _randn(g, E, D, std=0.02), torch.zeros(E, device=DEV), 1, 1, k, True, 1.0)
    y4 = _run(x, w, idx, tw).float()
    sh = moe.moe_dequantize(*w["sh_gate_up"])
    y16 = moe.moe_forward(x, moe.moe_dequantize(*w["gate_up"]), moe.moe_dequantize(*w["down"]),
                          sh[:d].contiguous(), sh[d:].contiguous(), moe.moe_dequantize(*w["sh_down"]),
                          idx, tw).float()
    assert moe.moe_device_status() == 0
    assert ((y4 - y16).norm() / y16.norm()).item() < 4 * 2.0 ** -8


def test_prompt_path_by_grouped_products():
    """The layer put together from its parts for a long batch: dequantize, sort the pairs by
    expert, two grouped products, weighted sum; the same output as the 4-bit layer."""
    N, D, E, k, d = 200, 256, 8, 4, 128
    x, w, ids, tw = _layer(N, D, E, k, d, d, 64, seed=11)
    order = torch.sort(ids.flatten().long(), stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.bincount(order.values, minlength=E).cumsum(0)
    tok = order.indices // k
    gu = moe.moe_grouped_linear(x[tok], moe.moe_dequantize(*w["gate_up"]), off)
    h = (torch.nn.functional.silu(gu[:, :d].float()) * gu[:, d:].float()).to(BF16)
    o = moe.moe_grouped_linear(h, moe.moe_dequantize(*w["down"]), off).float()
    y = torch.zeros((N, D), device=DEV).index_add_(0, tok, o * tw.flatten()[order.indices][:, None])
    s = moe.moe_linear_quant(x, *w["sh_gate_up"])
    s = (torch.nn.functional.silu(s[:, :d].float()) * s[:, d:].float()).to(BF16)
    y += moe.moe_linear_quant(s, *w["sh_down"]).float()
    got = _run(x, w, ids, tw).float()
    assert moe.moe_device_status() == 0
    assert ((got - y).norm() / y.norm()).item() < 4 * 2.0 ** -8


@pytest.mark.parametrize("N", [1, 24])
def test_layer_in_a_graph_with_new_routing(N):
    x, w, ids, tw = _layer(N, 256, 6, 2, 128, 128, 64, seed=6)
    ws = torch.empty(moe.moe_forward_quant_workspace(N, 256, 6, 128, 128, 2), dtype=torch.uint8, device=DEV)
    y = torch.empty_like(x)
    _run(x, w, ids, tw, y=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(x, w, ids, tw, y=y, workspace=ws)
    for shift in (0, 1, 3):
        ids.copy_((ids + shift) % 6)
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, _run(x, w, ids, tw))


def test_calls_in_a_row_on_one_stream_need_no_gap():
    """The kernels start before their predecessors end: a chain of calls, each reading the
    last one's output, gives what calls with a synchronisation between them give."""
    g = _gen(8)
    ws = [moe.moe_quantize(_randn(g, 256, 256, std=0.06), 32) for _ in range(6)]
    x = _randn(g, 4, 256)
    want = x
    for w in ws:
        want = moe.moe_linear_quant(want, *w)
        torch.cuda.synchronize()
    for _ in range(20):
        y = x
        for w in ws:
            y = moe.moe_linear_quant(y, *w)
        assert torch.equal(y, want)


def test_refusals():
    g = _gen(0)
    W = _randn(g, 64, 256)
    q, s = moe.moe_quantize(W, 64)
    x = _randn(g, 3, 256)
    for bad in (lambda: moe.moe_quantize(W.float(), 64), lambda: moe.moe_quantize(W, 48),
                lambda: moe.moe_quantize(W[:, :96], 64), lambda: moe.moe_quantize(W.cpu(), 64),
                lambda: moe.moe_quantize(W.t(), 32), lambda: moe.moe_linear_quant(x.float(), q, s),
                lambda: moe.moe_linear_quant(x[:, :128], q, s), lambda: moe.moe_linear_quant(x, q, s.t()),
                lambda: moe.moe_linear_quant(x, q, s[:, :32]), lambda: moe.moe_linear_quant(x, q.cpu(), s),
                lambda: moe.moe_linear_quant(x, q, s, y=torch.empty_like(x)),
                lambda: moe.moe_dequantize(q, s.float()), lambda: moe.moe_dequantize(q[None], s)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoEError):   # rows not a multiple of 8
        moe.moe_linear_quant(x, q[:60].contiguous(), s[:, :60].contiguous())
    x, w, ids, tw = _layer(4, 256, 6, 2, 128, 128, 64)
    with pytest.raises(ValueError):
        _run(x, w, ids.long(), tw)
    with pytest.raises(ValueError):
        _run(x, {**w, "down": moe.moe_quantize(_randn(g, 6, 256, 128), 32)}, ids, tw)
    with pytest.raises(moe.MoEError):
        _run(x, w, ids, tw, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(moe.MoEError):
        _run(x, w, ids, tw, gate_max=float("nan"))
    assert moe.moe_linear_quant(x[:0], *w["sh_gate_up"]).shape == (0, 256)
    assert _run(x[:0], w, ids[:0], tw[:0]).shape == (0, 256)


@pytest.mark.parametrize("N", [1, 5, 20, 97])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_device_usable(N):
    g = _gen(N)
    q, s = moe.moe_quantize(_randn(g, 1024, 4096, std=0.02), 64)
    xl = _randn(g, N, 4096)
    x, w, ids, tw = _layer(N, 512, 6, 2, 512, 256, 64)
    calls = lambda: (moe.moe_linear_quant(xl, q, s), _run(x, w, ids, tw))
    want = calls()
    assert moe.moe_device_status() == 0
    try:
        moe.moe_debug_set_wait_limit_ns(1)
        for _ in range(3):
            calls()
            assert moe.moe_device_status() in (0, -6)
    finally:
        moe.moe_debug_set_wait_limit_ns(0)
    for a, b in zip(calls(), want):
        assert torch.equal(a, b)
    assert moe.moe_device_status() == 0


def test_offsets_past_32_bits():
    """More than 2^31 weights: the last matrix is converted like one by itself."""
    E = 2 ** 31 // (1024 * 4096) + 1
    W = torch.zeros((E, 1024, 4096), dtype=BF16, device=DEV)
    W[-1] = _randn(_gen(0), 1024, 4096, std=0.02)
    q, s = moe.moe_quantize(W, 128)
    q1, s1 = moe.moe_quantize(W[-1], 128)
    assert torch.equal(q[-1], q1) and torch.equal(s[-1], s1)
    assert (q[:-1] == 0x88).all() and (s[:-1] == 0).all()
    back = moe.moe_dequantize(q, s, W=W)
    assert torch.equal(back[-1], moe.moe_dequantize(q1, s1)) and (back[:-1] == 0).all()


@pytest.mark.parametrize("N,M,K,G", [(96, 128, 128, 128), (97, 136, 256, 32), (192, 264, 640, 64),
                                     (193, 40, 384, 128), (300, 1000, 96, 32), (24, 4104, 64, 64)])
def test_product_with_many_tokens(N, M, K, G):
    g = _gen(N + M)
    q, s = moe.moe_quantize(_randn(g, M, K, std=0.02), G)
    x = _randn(g, N, K)
    w = _values(q, s)
    y = x.double() @ w.t()
    bad = ~((moe.moe_linear_quant(x, q, s).double() - y).abs() <= _product_tol(x, w, K, y))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    assert moe.moe_device_status() == 0


def test_large_tokens():
    """Tokens up to 2^62 and scales up to 2^50 are finite numbers like others."""
    g = _gen(3)
    q, s = moe.moe_quantize(_randn(g, 64, 256), 64)
    x = _randn(g, 4, 256)
    want = moe.moe_linear_quant(x, q, s)
    assert torch.equal(moe.moe_linear_quant(x * 2.0 ** 60, q, s), want * 2.0 ** 60)
    assert torch.equal(moe.moe_linear_quant(x * 2.0 ** -60, q, s), want * 2.0 ** -60)
    assert torch.equal(moe.moe_linear_quant(x, q, s * 2.0 ** 50), want * 2.0 ** 50)


def test_two_streams_at_once():
    g = _gen(12)
    ws = [moe.moe_quantize(_randn(g, 512, 1024, std=0.02), 64), moe.moe_quantize(_randn(g, 2048, 256, std=0.02), 32)]
    xs = [_randn(g, 40, 1024), _randn(g, 3, 256)]
    want = [moe.moe_linear_quant(x, *w) for x, w in zip(xs, ws)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[moe.moe_linear_quant(xs[i], *ws[i], y=torch.empty_like(want[i]), stream=streams[i])
            for i in range(2)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(y[i], want[i]) for y in got for i in range(2))


def test_what_a_call_makes_is_memory_of_the_calls_stream():
    # The current stream gives a block back while its last write is still to come; a call on
    # another stream must not be handed that block.
    g = _gen(13)
    W = _randn(g, 2048, 512, std=0.02)
    q, s = moe.moe_quantize(W, 64)
    x = _randn(g, 300, 512)
    other = torch.cuda.Stream()
    for f in (lambda **k: moe.moe_linear_quant(x, q, s, **k), lambda **k: moe.moe_dequantize(q, s, **k)):
        want = f()
        for stream in (other, other.cuda_stream):
            torch.cuda.synchronize()
            scratch = torch.empty_like(want)
            torch.cuda._sleep(100_000_000)
            scratch.fill_(float("nan"))
            del scratch
            got = f(stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    x, w, ids, tw = _layer(12, 256, 6, 2, 128, 128, 64)
    want = _run(x, w, ids, tw)
    torch.cuda.synchronize()
    got = [_run(x, w, ids, tw, stream=other) for _ in range(4)]  # workspaces taken and given back there
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


# Columns shared by the blocks of a cluster, for one row tile and for more tiles than
# clusters; columns that end inside a stage of 128; token counts that no share divides.
@pytest.mark.parametrize("N,M,K,G", [(17, 264, 1024, 64), (96, 8, 896, 64), (33, 40, 8192, 128), (90, 1032, 2208, 32),
                                     (20, 2816, 4096, 32), (200, 520, 1504, 32), (77, 12288, 2048, 64),
                                     (40, 24576, 1024, 128), (81, 12288, 5120, 32)])
def test_product_of_many_tokens_in_clusters(N, M, K, G):
    g = _gen(N + M + K)
    q, s = moe.moe_quantize(_randn(g, M, K, std=0.02), G)
    x = _randn(g, N, K)
    w = _values(q, s)
    y = x.double() @ w.t()
    tol = _product_tol(x, w, K, y)
    first = moe.moe_linear_quant(x, q, s)
    for _ in range(3):
        got = moe.moe_linear_quant(x, q, s)
        bad = ~((got.double() - y).abs() <= tol)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
        assert torch.equal(got, first)
    assert moe.moe_device_status() == 0
