"""Products grouped by expert: the experts' linear maps one by one, with gradients.

    y = moe_grouped_linear(x, W, offsets)          # rows [offsets[e], offsets[e+1]) times W[e]^T
    dx = moe_grouped_linear_dgrad(dy, W, offsets)
    dW = moe_grouped_linear_wgrad(dy, x, offsets)

moe_grouped_linear takes part in autograd.  Every call runs on the tensors' own device,
on that device's current stream unless a stream is given, and needs all tensors there.
What a call makes belongs, as torch's allocator sees it, to the stream the call runs on.
"""

from __future__ import annotations

import torch

from . import MOE_BF16, MOE_F32, _check, load_library

__all__ = ["moe_grouped_linear", "moe_grouped_linear_dgrad", "moe_grouped_linear_wgrad"]


# The calls themselves take a few microseconds on the GPU at decode sizes, so what a binding
# spends before the launch is kept small: a tensor's device is read as an index, the current
# stream as a raw handle, and the device is switched only where it differs.
_current_stream = torch._C._cuda_getCurrentRawStream
_DTYPES = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}


def _dt(t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)
    return code


def _device(*tensors):
    """The index of the device all tensors are on; they must be contiguous."""
    dev = -2
    for t in tensors:
        if not isinstance(t, torch.Tensor) or t.get_device() != dev:
            if dev != -2 or not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError("the tensors must be CUDA tensors on one device")
            dev = t.get_device()
        if not t.is_contiguous():
            raise ValueError("the tensors must be contiguous")
    return dev


def _handle(stream):
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def _call(name, dev, stream, *args):
    """One library call on device dev, with the stream as its last argument."""
    f = getattr(load_library(), name)
    stream = _current_stream(dev) if stream is None else _handle(stream)
    if dev == torch.cuda.current_device():
        rc = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, stream)
    if rc:
        _check(rc, name)


def _new(shape, dtype, like, stream):
    """A tensor (unset) on the device of `like` for a call on `stream`.  It is taken from that
    stream's memory: a block that the current stream has given back may still be in use
    there, and one that this call gives back is still in use here."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(torch.cuda.ExternalStream(_handle(stream), device=like.device)):
        return like.new_empty(shape, dtype=dtype)


def _out(t, shape, dtype, like, name, stream):
    """An output the caller gave, checked, or a new one."""
    if t is None:
        return _new(shape, dtype, like, stream)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.get_device() != like.get_device() \
            or not t.is_contiguous():
        raise ValueError("%s must be contiguous, %s %s on the inputs' device" % (name, list(shape), dtype))
    return t


def _same_type(*ts):
    for t in ts[1:]:
        if t.dtype != ts[0].dtype:
            raise ValueError("the tensors must share one dtype")


def _check_sizes(rows, offsets, E):
    if rows > 0x7FFFFFFF:  # an int's, in the library
        raise ValueError("at most 2^31 - 1 rows")
    if offsets.dtype != torch.int32 or tuple(offsets.shape) != (E + 1,):
        raise ValueError("offsets must be int32 [E + 1]")


def _linear(x, W, offsets, y, stream):
    if x.dim() != 2 or W.dim() != 3 or W.shape[2] != x.shape[1]:
        raise ValueError("x must be [rows, K] and W [E, M, K]")
    dev = _device(x, W, offsets)
    _same_type(x, W)
    (rows, K), (E, M, _) = x.shape, W.shape
    _check_sizes(rows, offsets, E)
    rest = int(y is None)
    y = _out(y, (rows, M), x.dtype, x, "y", stream)
    _call("moe_grouped_linear", dev, stream, x.data_ptr(), W.data_ptr(), offsets.data_ptr(), rows,
          E, M, K, _dt(x), y.data_ptr(), rest)
    return y


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, offsets):
        ctx.save_for_backward(x, W, offsets)
        return _linear(x, W, offsets, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, W, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = moe_grouped_linear_dgrad(dy, W, offsets) if ctx.needs_input_grad[0] else None
        dW = moe_grouped_linear_wgrad(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dW, None


def _accumulation(leaf):
    """The notes (a dict) of the node that accumulates a leaf's gradient."""
    return torch.autograd.graph.get_gradient_edge(leaf).node.metadata


def _differentiable(x, W, offsets):
    """_GroupedLinear, refusing a capture on a leaf whose gradient accumulation belongs to an
    eager pass on the default stream.

    Autograd keeps one accumulation node per leaf while any pass (or a wrapper, such as a
    data-parallel one) holds it, tied to the stream it was made on.  A backward pass captured
    on another stream joins that stream: one that can be captured takes part, the default
    stream (handle 0) cannot, which ends the capture and the process.  So every call leaves
    its stream on the nodes it is the first to see, and a captured one reads it.  A node that
    something else made on the default stream, and that a call on another stream saw first,
    is not recognised."""
    leaves = [t.requires_grad and t.is_leaf for t in (x, W)]
    here = _current_stream(torch.cuda.current_device())
    if torch.cuda.is_current_stream_capturing():
        for t, leaf in zip((x, W), leaves):
            if leaf and _accumulation(t).get("moe_stream", here) == 0:
                raise ValueError("capturing: an eager pass over the same leaf tensors, made on the default "
                                 "stream, is still alive; drop its outputs first, or run it on another stream")
    y = _GroupedLinear.apply(x, W, offsets)
    for leaf, (node, _) in zip(leaves, y.grad_fn.next_functions):
        if leaf:
            node.metadata.setdefault("moe_stream", here)
    return y


def moe_grouped_linear(x, W, offsets, y=None, stream=None):
    """y [rows, M] with y_r = W[e] x_r for the rows r of expert e, offsets[e] <= r < offsets[e+1].

    x [rows, K] and W [E, M, K] bf16 or fp32, offsets int32 [E + 1], all contiguous on one
    device.  A y that is given keeps its rows of no expert; a new one has zeros there.
    Differentiable in x and W (rows of no expert have a zero gradient), without a y or a
    stream of the caller's; the backward pass runs on the stream autograd gives it."""
    if torch.is_grad_enabled() and (x.requires_grad or W.requires_grad):
        if y is not None or stream is not None:
            raise ValueError("y and stream: not with gradients (use torch.no_grad, torch.cuda.stream)")
        dev = _device(x, W, offsets)
        if dev == torch.cuda.current_device():
            return _differentiable(x, W, offsets)
        with torch.cuda.device(dev):
            return _differentiable(x, W, offsets)
    return _linear(x, W, offsets, y, stream)


def moe_grouped_linear_dgrad(dy, W, offsets, dx=None, stream=None):
    """dx [rows, K] with dx_r = W[e]^T dy_r, the gradient of moe_grouped_linear in x.
    A dx that is given keeps its rows of no expert; a new one has zeros there."""
    if dy.dim() != 2 or W.dim() != 3 or W.shape[1] != dy.shape[1]:
        raise ValueError("dy must be [rows, M] and W [E, M, K]")
    dev = _device(dy, W, offsets)
    _same_type(dy, W)
    rows, (E, M, K) = dy.shape[0], W.shape
    _check_sizes(rows, offsets, E)
    rest = int(dx is None)
    dx = _out(dx, (rows, K), dy.dtype, dy, "dx", stream)
    _call("moe_grouped_linear_dgrad", dev, stream, dy.data_ptr(), W.data_ptr(), offsets.data_ptr(),
          rows, E, M, K, _dt(dy), dx.data_ptr(), rest)
    return dx


def moe_grouped_linear_wgrad(dy, x, offsets, dW=None, stream=None):
    """dW [E, M, K] with dW[e] = sum over e's rows of dy_r x_r^T, the gradient of
    moe_grouped_linear in W (zeros for an expert without rows)."""
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0]:
        raise ValueError("dy must be [rows, M] and x [rows, K]")
    dev = _device(dy, x, offsets)
    _same_type(dy, x)
    (rows, M), K, E = dy.shape, x.shape[1], offsets.shape[0] - 1
    _check_sizes(rows, offsets, E)
    dW = _out(dW, (E, M, K), dy.dtype, dy, "dW", stream)
    _call("moe_grouped_linear_wgrad", dev, stream, dy.data_ptr(), x.data_ptr(), offsets.data_ptr(),
          rows, E, M, K, _dt(dy), dW.data_ptr())
    return dW
