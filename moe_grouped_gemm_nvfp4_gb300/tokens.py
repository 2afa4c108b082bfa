"""Token rows into expert order and back, with their gradients.

`dispatch` copies each token's row to its routes' positions, `combine` brings
the experts' rows back as the weighted sum of each token's routes; both take
part in autograd (the tokens', the experts' rows' and the routing weights'
gradients).  The positions are nvfp4.moe_route's: route_pos int32 [T, topk],
negative for a dropped route, and expert_offsets int32 [E + 1].  Rows are BF16,
FP16 or FP32 of any width; rows whose elements are not neighbours are copied
first, any other row stride is used as it is.

`dispatch_grad` and `combine_grad` are the gradients as plain calls, which take no
part in autograd; they enqueue kernels only, so that a step made of them can be
captured into a CUDA graph.  (A captured step should not run autograd's backward
over leaves that an eager graph still holds: torch binds a leaf's accumulation to
the stream of its first use.)  There is no forward-mode derivative: tensors that
carry a tangent are refused.

Work goes to the current stream of the tensors' device, whichever device is
current, or to `stream` (a torch stream of that device or a raw handle), where the
outputs are then allocated too.  The arithmetic runs in the
CUDA kernels; sums are FP32 in a fixed order.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from .nvfp4 import native


def on_stream(stream, device):
    """Context that makes `stream` (a torch stream or a raw handle) of the tensors'
    `device` current there, so that the calls find it and memory freed on return is
    reused in that stream's order."""
    if device.type != "cuda":
        raise ValueError("expected a CUDA tensor")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device != device:
        raise ValueError(f"stream: of {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def refuse_tangents(*tensors):
    """Forward-mode tangents would be lost (the derivative zero) without an error;
    `requires_grad` does not show them.  The calls come here only while a dual level
    is open (forward_ad._current_level >= 0): a whole call of one token takes 5 us."""
    if any(isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None
           for t in tensors):
        raise RuntimeError("no forward-mode derivative: a tensor carries a tangent")


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, route_pos, expert_offsets, R):
        ctx.save_for_backward(route_pos)
        return native().dispatch(x, route_pos, expert_offsets, R, True)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        return native().combine(dout, ctx.saved_tensors[0], None), None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, route_pos, weights, expert_offsets):
        ctx.save_for_backward(y, route_pos, weights,
                              *([] if expert_offsets is None else [expert_offsets]))
        return native().combine(y, route_pos, weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        y, route_pos, weights, *offsets = ctx.saved_tensors
        if weights is None:
            weights = torch.ones(route_pos.shape, dtype=torch.float32, device=y.device)
        dy, dw = native().combine_grad(dout, y, route_pos, weights,
                                       offsets[0] if offsets else None, True)
        return dy, None, dw if ctx.needs_input_grad[2] else None, None


def dispatch(x, route_pos, expert_offsets=None, R=None, stream=None):
    """x [T, D] -> rows in expert order [R, D] (R: T * topk unless given).  Rows
    past expert_offsets[E] are zero.  Without expert_offsets, rows that no route
    names are zero while torch records gradients (an expert's weight gradient
    sums over every row, and zero times stale memory may be NaN), which costs a
    fill of the buffer, and are left unwritten under no_grad."""
    if forward_ad._current_level >= 0:
        refuse_tangents(x)
    R = -1 if R is None else R
    if stream is not None:
        with on_stream(stream, x.device):
            return dispatch(x, route_pos, expert_offsets, R)
    if x.requires_grad and torch.is_grad_enabled():
        return _Dispatch.apply(x, route_pos, expert_offsets, R)
    return native().dispatch(x, route_pos, expert_offsets, R, torch.is_grad_enabled())


def dispatch_grad(dout, route_pos, stream=None):
    """Gradient of `dispatch`: dout [R, D] -> [T, D], the sum over each token's
    routes."""
    if forward_ad._current_level >= 0:
        refuse_tangents(dout)
    if stream is not None:
        with on_stream(stream, dout.device):
            return native().combine(dout, route_pos, None)
    return native().combine(dout, route_pos, None)


def combine(y, route_pos, weights=None, expert_offsets=None, stream=None):
    """y [R, D] in expert order -> [T, D]: the sum of each token's routes, times
    weights (FP32 [T, topk]) where given.  The gradient's rows that no route names
    are zero; expert_offsets, which only the backward pass uses, lets it zero the
    rows past expert_offsets[E] instead of filling the whole buffer first."""
    if forward_ad._current_level >= 0:
        refuse_tangents(y, weights)
    if stream is not None:
        with on_stream(stream, y.device):
            return combine(y, route_pos, weights, expert_offsets)
    if (y.requires_grad or (weights is not None and weights.requires_grad)) \
            and torch.is_grad_enabled():
        return _Combine.apply(y, route_pos, weights, expert_offsets)
    return native().combine(y, route_pos, weights)


def combine_grad(dout, y, route_pos, weights, expert_offsets=None, stream=None):
    """Gradient of `combine`: (dy [R, D], dweights FP32 [T, topk]).  Rows of dy
    past expert_offsets[E] are zero; without expert_offsets, rows that no route
    names are left unwritten."""
    if forward_ad._current_level >= 0:
        refuse_tangents(dout, y, weights)
    if stream is not None:
        with on_stream(stream, y.device):
            return native().combine_grad(dout, y, route_pos, weights, expert_offsets, False)
    return native().combine_grad(dout, y, route_pos, weights, expert_offsets, False)
