"""Weights in 4 bits with group scales, and the products that read them.

    q, scales = moe_quantize(W, group)             # W [..., M, K] bf16
    W = moe_dequantize(q, scales)
    y = moe_linear_quant(x, q, scales)             # x [N, K] bf16, q [M, K/2]
    y = moe_forward_quant(x, gate_up, down, sh_gate_up, sh_down, topk_idx, topk_w)

A matrix [M, K] is a pair (q, scales): q uint8 [M, K/2], column 2j in the low and 2j + 1 in
the high four bits of byte j, scales bf16 [K/group, M]; its value at (m, k) is
(code - 8) * scales[k // group, m].  The group size is read off the shapes.
Every call runs on the tensors' own device, on that device's current stream unless a
stream is given, and needs all tensors there.  What a call makes belongs, as torch's
allocator sees it, to the stream the call runs on.  No call takes part in autograd.
"""

from __future__ import annotations

import torch

from . import load_library
from .products import _call, _device, _new, _out

__all__ = ["moe_quantize", "moe_dequantize", "moe_linear_quant", "moe_forward_quant",
           "moe_forward_quant_workspace"]


def _pair(q, scales, lead, name):
    """(M, K, group) of 4-bit weights with `lead` leading dimensions."""
    if q.dtype != torch.uint8 or scales.dtype != torch.bfloat16:
        raise ValueError("%s must be (uint8 codes, bfloat16 scales)" % name)
    qs, ss = q.shape, scales.shape
    if lead >= 0 and len(qs) == lead + 2 and len(ss) == lead + 2 and qs[:lead] == ss[:lead]:
        M, K, groups = qs[lead], 2 * qs[lead + 1], ss[lead]
        if ss[lead + 1] == M and groups and not K % groups:
            return M, K, K // groups
    raise ValueError("%s: codes [.., M, K/2] and scales [.., K/group, M] do not agree" % name)


def moe_quantize(W, group: int = 128, q=None, scales=None, stream=None):
    """(q, scales) of bf16 weights W [..., M, K], group = 32, 64 or 128."""
    if W.dim() < 2 or W.dtype != torch.bfloat16:
        raise ValueError("W must be bfloat16 [..., M, K]")
    dev = _device(W)
    lead, (M, K) = tuple(W.shape[:-2]), W.shape[-2:]
    if group not in (32, 64, 128) or K % group:
        raise ValueError("group must be 32, 64 or 128 and divide K")
    q = _out(q, lead + (M, K // 2), torch.uint8, W, "q", stream)
    scales = _out(scales, lead + (K // group, M), torch.bfloat16, W, "scales", stream)
    E = W.numel() // (M * K) if M * K else 0
    _call("moe_quantize", dev, stream, W.data_ptr(), E, M, K, group, q.data_ptr(), scales.data_ptr())
    return q, scales


def moe_dequantize(q, scales, W=None, stream=None):
    """The bf16 values [..., M, K] of 4-bit weights."""
    M, K, group = _pair(q, scales, q.dim() - 2, "the weights")
    dev = _device(q, scales)
    W = _out(W, tuple(q.shape[:-2]) + (M, K), torch.bfloat16, q, "W", stream)
    E = W.numel() // (M * K) if M * K else 0
    _call("moe_dequantize", dev, stream, q.data_ptr(), scales.data_ptr(), E, M, K, group, W.data_ptr())
    return W


def moe_linear_quant(x, q, scales, y=None, stream=None):
    """y [N, M] = x W^T for tokens x [N, K] bf16 and one matrix in 4 bits."""
    M, K, group = _pair(q, scales, 0, "the weights")
    if x.dim() != 2 or x.shape[1] != K or x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16 [N, K]")
    dev = _device(x, q, scales)
    N = x.shape[0]
    y = _out(y, (N, M), torch.bfloat16, x, "y", stream)
    _call("moe_linear_quant", dev, stream, x.data_ptr(), q.data_ptr(), scales.data_ptr(), N, M, K,
          group, y.data_ptr())
    return y


def moe_forward_quant_workspace(N: int, D: int, E: int, d_moe: int, d_sh: int, k: int) -> int:
    """Bytes of device workspace moe_forward_quant needs (0 for invalid sizes)."""
    return int(load_library().moe_forward_quant_workspace(N, D, E, d_moe, d_sh, k))


def moe_forward_quant(x, gate_up, down, sh_gate_up, sh_down, topk_idx, topk_w, y=None,
                      workspace=None, stream=None, gate_max=None, up_max=None):
    """moe_forward with all experts in 4 bits; returns y [N, D] bf16.

    gate_up, down, sh_gate_up, sh_down: (q, scales) pairs of [E, 2 d_moe, D] (gate rows
    first), [E, D, d_moe], [2 d_sh, D] (gate rows first) and [D, d_sh], one group size.
    topk_idx [N, k] int32 (id E: no expert), topk_w [N, k] fp32.  gate_max / up_max: the
    clamped SwiGLU's limits."""
    two_d, D, group = _pair(*gate_up, 1, "gate_up")
    D2, d, g2 = _pair(*down, 1, "down")
    two_ds, D3, g3 = _pair(*sh_gate_up, 0, "sh_gate_up")
    D4, d_sh, g4 = _pair(*sh_down, 0, "sh_down")
    E = gate_up[0].shape[0]
    if x.dim() != 2 or x.shape[1] != D or x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16 [N, D]")
    if (D2, D3, D4) != (D, D, D) or two_d != 2 * d or two_ds != 2 * d_sh \
            or down[0].shape[0] != E or (g2, g3, g4) != (group,) * 3:
        raise ValueError("inconsistent expert shapes or group sizes")
    N = x.shape[0]
    if topk_idx.dim() != 2 or topk_idx.shape[0] != N or topk_w.shape != topk_idx.shape \
            or topk_idx.dtype != torch.int32 or topk_w.dtype != torch.float32:
        raise ValueError("topk_idx must be int32 and topk_w float32, both [N, k]")
    k = topk_idx.shape[1]
    dev = _device(x, *gate_up, *down, *sh_gate_up, *sh_down, topk_idx, topk_w)
    y = _out(y, (N, D), torch.bfloat16, x, "y", stream)
    if workspace is None:
        workspace = _new((max(moe_forward_quant_workspace(N, D, E, d, d_sh, k), 256),),
                         torch.uint8, x, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous, on the inputs' device")
    inf = float("inf")
    _call("moe_forward_quant", dev, stream, x.data_ptr(), gate_up[0].data_ptr(),
          gate_up[1].data_ptr(), down[0].data_ptr(), down[1].data_ptr(), sh_gate_up[0].data_ptr(),
          sh_gate_up[1].data_ptr(), sh_down[0].data_ptr(), sh_down[1].data_ptr(),
          topk_idx.data_ptr(), topk_w.data_ptr(), N, D, E, d, d_sh, k, group,
          inf if gate_max is None else float(gate_max), inf if up_max is None else float(up_max),
          y.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return y
