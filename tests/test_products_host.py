"""Host-side refusals of the products by expert and of the 4-bit layer (no GPU)."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_moe_layer_02_b200 as moe


def test_no_workspace_for_a_layer_that_is_refused():
    """moe_forward_quant_workspace is 0 exactly where moe_forward_quant refuses the sizes for every
    group (16: pointers that pass the alignment check; the refusal comes before any use)."""
    lib = moe.load_library()

    def both(N=4, D=256, E=8, d=128, d_sh=128, k=2):
        sizes = [N, D, E, d, d_sh, k]
        w = lib.moe_forward_quant_workspace(*sizes)
        refused = all(lib.moe_forward_quant(*[16] * 11, *sizes, G, 1.0, 1.0, 16, None, 0, None) == -2
                      for G in (32, 64, 128))
        return w, refused
    for bad in (dict(N=-1), dict(N=(1 << 24) + 1), dict(D=250), dict(D=0), dict(D=1 << 21), dict(d=40), dict(d=0),
                dict(d_sh=16), dict(d=1 << 20), dict(E=0), dict(E=513), dict(k=0), dict(k=33),
                dict(N=1 << 24, D=1 << 20, d=1 << 19, k=32)):
        assert both(**bad) == (0, True), bad
    for good in (dict(), dict(D=32, d=32, d_sh=32), dict(N=0), dict(N=1), dict(N=100000, D=6144, E=256, d=2048)):
        w, refused = both(**good)
        assert w > 0 and not refused, good


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32 + 5])
def test_more_rows_than_an_int_counts_are_refused(rows):
    """Tensors without memory: the library's argument would wrap (2^32 + 5 rows to 5)."""
    with FakeTensorMode():
        t = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")
        x, W, off, dy = t(rows, 8), t(2, 16, 8), t(3, dtype=torch.int32), t(rows, 16)
        for f in (lambda: moe.moe_grouped_linear(x, W, off), lambda: moe.moe_grouped_linear_dgrad(dy, W, off),
                  lambda: moe.moe_grouped_linear_wgrad(dy, x, off)):
            with pytest.raises(ValueError, match="rows"):
                f()
