"""The products with 4-bit weights over the range of their tokens and codes, for token counts on
both sides of the choices between kernels and tiles.

Tolerances.  (code - 8) * token is exact in fp32 (4 + 8 bits).  A tensor-core step of 16 products
is taken to lose at most 2^-22 of its largest partial sum, and a group's multiply-add and the
sums of slices and blocks 2^-24 each, so (K/16 + K/32 + 10) * 2^-22 of S = sum |x w| bounds what a
sum loses; y is rounded once to bf16 (2^-8 of its value).  S counts a column coded 8 as nothing,
whatever its token.  A row with one code other than 8 has one product, of 4 + 8 + 8 bits, exact
in fp32: y is its one rounding, whatever the other tokens are.  Powers of two only shift exponents.
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


def _check(got, x, w):
    y, mass, K = x.double() @ w.t(), x.double().abs() @ w.abs().t(), x.shape[1]
    tol = y.abs() * 2.0 ** -8 + mass * (K / 16 + K / 32 + 10) * 2.0 ** -22
    bad = ~((got.double() - y).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), y[bad][:4].tolist())


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N", [1, 8, 16, 17, 24, 25, 33, 50])
def test_tokens_and_scales_of_any_size(N, G):
    g = _gen(N + G)
    q, s = moe.moe_quantize(_randn(g, 264, 1024, std=0.02), G)
    x = _randn(g, N, 1024)
    want = moe.moe_linear_quant(x, q, s)
    _check(want, x, _values(q, s))
    for p in (-110, -90, -70, 64, 90, 110):
        assert torch.equal(moe.moe_linear_quant(x * 2.0 ** p, q, s), want * 2.0 ** p), p
    for p in (-100, -60, 60, 100, 120):
        assert torch.equal(moe.moe_linear_quant(x, q, s * 2.0 ** p), want * 2.0 ** p), p


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N", [8, 16, 17, 25, 33, 50])
def test_tokens_below_the_normal_numbers(N, G):
    """Tokens around 2^-126 with large scales: nothing is flushed to zero on the way."""
    g = _gen(N + G)
    q, s = moe.moe_quantize(_randn(g, 136, 512, std=0.02), G)
    s = s * 2.0 ** 60
    x = _randn(g, N, 512) * 2.0 ** -124
    got = moe.moe_linear_quant(x, q, s)
    _check(got, x, _values(q, s))


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N", [1, 8, 16, 17, 24, 25, 33, 50])
def test_columns_coded_zero_leave_no_residue(N, G):
    """Rows with one weight other than 0, on columns of small tokens; large tokens elsewhere."""
    g = _gen(3 * N + G)
    M, K = 200, 768
    col = torch.randint(0, K // 2, (M,), generator=g, device=DEV) * 2
    code = torch.randint(0, 8, (M,), generator=g, device=DEV)     # -8 .. -1
    code = torch.where(torch.rand(M, generator=g, device=DEV) < 0.5, code, 16 - 1 - code)
    q = torch.full((M, K // 2), 0x88, dtype=torch.uint8, device=DEV)
    q[torch.arange(M, device=DEV), col // 2] = (code | 0x80).to(torch.uint8)
    s = _randn(g, K // G, M)
    x = _randn(g, N, K)
    x[:, 1::2] *= 2.0 ** 30
    x[:, ::4] *= 2.0 ** -10
    rows = torch.arange(M, device=DEV)
    want = x[:, col].double() * (code.double() - 8.0) * s[col // G, rows].double()
    assert torch.equal(moe.moe_linear_quant(x, q, s), want.to(BF16))


@pytest.mark.parametrize("N", [1, 6, 40])
def test_layer_with_small_tokens(N):
    """Small tokens make the SwiGLU output very small (about the square): gate and up near 2^-45,
    their product near 2^-91.  silu(a) = a / 2 there, up to a^2 / 4 < 2^-90 of it."""
    g = _gen(N)
    D, E, k, d = 256, 6, 2, 128
    pair = lambda *shape: moe.moe_quantize(_randn(g, *shape, std=0.05), 64)
    gu, dn, sgu, sdn = pair(E, 2 * d, D), pair(E, D, d), pair(2 * d, D), pair(D, d)
    x = _randn(g, N, D) * 2.0 ** -45
    ids = torch.rand((N, E), generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
    tw = torch.rand((N, k), generator=g, device=DEV)
    got = moe.moe_forward_quant(x, gu, dn, sgu, sdn, ids, tw)
    # the same layer with tokens that are 1 / 2^45: gate and up linear in x, h quadratic; to keep
    # silu(a) = a / 2 exact, the oracle is written for small a
    def expert(rows, gu, dn):
        a, u = (x[rows].double() @ gu.t()).chunk(2, dim=1)
        ma, mu = (x[rows].double().abs() @ gu.abs().t()).chunk(2, dim=1)
        h = a / 2 * u
        f, fd = (D / 16 + D / 32 + 10) * 2.0 ** -22, (d / 16 + d / 32 + 10) * 2.0 ** -22
        dh = (ma * f * (u.abs() + mu * f) + mu * f * a.abs()) / 2 + h.abs() * (2.0 ** -8 + 2.0 ** -20) * 1.01
        return h @ dn.t(), (dh + h.abs() * fd) @ dn.abs().t()
    y, tol = expert(slice(None), _values(*sgu), _values(*sdn))
    for e in range(E):
        rows, slots = (ids == e).nonzero(as_tuple=True)
        if len(rows):
            o, t = expert(rows, _values(gu[0][e], gu[1][e]), _values(dn[0][e], dn[1][e]))
            c = tw[rows, slots].double()[:, None]
            y.index_add_(0, rows, o * c)
            tol.index_add_(0, rows, t * c + (o * c).abs() * 8 * 2.0 ** -24)
    tol += y.abs() * 2.0 ** -8 * 1.01
    assert ((got.double() - y).abs() <= tol).all()
    assert moe.moe_device_status() == 0
