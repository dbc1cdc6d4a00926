"""4-bit products of very many tokens (offsets past 32 bits), and layers on two streams at once.

Tolerances as in the other tests of these products (S = sum |x w|): sums lose at most
(K/16 + K/32 + 10) * 2^-22 of S, an output is rounded once (2^-8 of its value), the SwiGLU
output too (with 2^-20 for its exponential and division), which weighs |down| |h|.
"""

import pytest
import torch

import sparse_moe_layer_02_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(BF16)


def _values(q, s):
    c = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).double() - 8.0
    return c * s.double().transpose(-1, -2).repeat_interleave(c.shape[-1] // s.shape[-2], dim=-1)


def _loss(K):
    return (K / 16 + K / 32 + 10) * 2.0 ** -22


def test_product_with_offsets_past_32_bits():
    """More than 2^31 outputs: the first and the last tokens, among many that are zero."""
    g = _gen(0)
    N, M, K = 131075, 16392, 128
    q, s = moe.moe_quantize(_randn(g, M, K, std=0.02), 128)
    x = torch.zeros((N, K), dtype=BF16, device=DEV)
    rows = torch.cat((torch.arange(40, device=DEV), torch.arange(N - 200, N, device=DEV)))
    x[rows] = _randn(g, 240, K)
    y = moe.moe_linear_quant(x, q, s)
    w = _values(q, s)
    want = x[rows].double() @ w.t()
    tol = want.abs() * 2.0 ** -8 + (x[rows].double().abs() @ w.abs().t()) * _loss(K)
    assert ((y[rows].double() - want).abs() <= tol).all()
    assert (y[40:-200] == 0).all()
    assert moe.moe_device_status() == 0


def _layer(g, N, D, E, k, d, G):
    pair = lambda *shape: moe.moe_quantize(_randn(g, *shape, std=0.05), G)
    w = pair(E, 2 * d, D), pair(E, D, d), pair(2 * d, D), pair(D, d)
    x = _randn(g, N, D)
    ids = torch.rand((N, E), generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
    return x, w, ids, torch.rand((N, k), generator=g, device=DEV)


def test_layer_with_offsets_past_32_bits():
    """N * k * D past 2^31: the kept outputs of the experts, and the last tokens' sums."""
    N, D, E, k, d = 70001, 4096, 8, 8, 64
    x, w, ids, tw = _layer(_gen(1), N, D, E, k, d, 64)
    got = moe.moe_forward_quant(x, *w, ids, tw)
    assert moe.moe_device_status() == 0
    rows = torch.cat((torch.arange(20, device=DEV), torch.arange(N - 60, N, device=DEV)))
    xd, (gu, dn, sgu, sdn) = x[rows].double(), w

    def expert(gu, dn):
        v, m = xd @ gu.t(), (xd.abs() @ gu.abs().t()) * _loss(D)
        a, u = v.chunk(2, dim=1)
        ea, eu = m.chunk(2, dim=1)
        h = a * torch.sigmoid(a) * u
        dh = 1.1 * ea * (u.abs() + eu) + eu * a.abs().clamp(min=1.0) + h.abs() * (2.0 ** -8 + 2.0 ** -20) * 1.01
        return h @ dn.t(), (dh + h.abs() * _loss(d)) @ dn.abs().t()
    y, tol = expert(_values(*sgu), _values(*sdn))
    for e in range(E):
        c = (tw[rows].double() * (ids[rows] == e)).sum(1, keepdim=True)
        o, t = expert(_values(gu[0][e], gu[1][e]), _values(dn[0][e], dn[1][e]))
        y += o * c
        tol += t * c + (o * c).abs() * 8 * 2.0 ** -24
    tol += y.abs() * 2.0 ** -8 * 1.01
    assert ((got[rows].double() - y).abs() <= tol).all()
    assert torch.equal(got, moe.moe_forward_quant(x, *w, ids, tw))


@pytest.mark.parametrize("Ns", [(1, 1), (1, 40), (6, 20)])
def test_layers_on_two_streams_at_once(Ns):
    cases = [_layer(_gen(i), N, 512, 12, 4, 256, 64) for i, N in enumerate(Ns)]
    call = lambda c, **kw: moe.moe_forward_quant(c[0], *c[1], c[2], c[3], **kw)
    want = [call(c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[call(c, stream=s) for c, s in zip(cases, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys in got for y, w in zip(ys, want))
    assert moe.moe_device_status() == 0
