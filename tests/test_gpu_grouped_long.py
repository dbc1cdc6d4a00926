"""Weight gradients over long segments: tens of thousands of rows of ordinary size.

Tolerances as in the other tests of these products: an fp32 result is one chain of n fused
multiply-adds, off by at most n * 2^-24 of sum |a b|; a bf16 one is rounded once (2^-8) after
sums that lose at most 2^-22 of the largest partial sum per 16 products, and 7 additions of
2^-24 where 8 blocks share them.
"""

import pytest
import torch

import sparse_moe_layer_02_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,M,K", [([40000, 0, 25001], 64, 40), ([70003], 32, 32), ([3, 50000], 200, 136)])
def test_weight_gradient_over_long_segments(sizes, M, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(M)
    rows = sum(sizes)
    x = torch.randn((rows, K), generator=g, device=DEV).to(dtype)
    dy = (torch.randn((rows, M), generator=g, device=DEV) + 0.5).to(dtype)  # a mean: sums that grow
    off = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    got = moe.moe_grouped_linear_wgrad(dy, x, off)
    a = 0
    for e, n in enumerate(sizes):
        d, v = dy[a:a + n].double(), x[a:a + n].double()
        exact, mass = d.t() @ v, d.abs().t() @ v.abs()
        if dtype == torch.float32:
            tol = mass * (n + 1) * 2.0 ** -24
        else:
            tol = exact.abs() * 2.0 ** -8 + mass * (n / 16 + 3) * 2.0 ** -22 * (1 + 2.0 ** -8)
        assert ((got[e].double() - exact).abs() <= tol).all()
        a += n
    assert torch.equal(got, moe.moe_grouped_linear_wgrad(dy, x, off))
    assert moe.moe_device_status() == 0
