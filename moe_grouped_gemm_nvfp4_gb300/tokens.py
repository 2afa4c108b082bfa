"""Token rows into expert order and back, with their gradients.

`dispatch` copies each token's row to its routes' positions, `combine` brings
the experts' rows back as the weighted sum of each token's routes; both take
part in autograd (the tokens', the experts' rows' and the routing weights'
gradients).  The positions are nvfp4.moe_route's: route_pos int32 [T, topk],
negative for a dropped route, and expert_offsets int32 [E + 1].  Rows are BF16,
FP16 or FP32 of any width and row stride.

`dispatch_grad` and `combine_grad` are the gradients as plain calls; they
enqueue kernels only, so that a step made of them can be captured into a CUDA
graph.  (A captured step should not run autograd's backward over leaves that an
eager graph still holds: torch binds a leaf's accumulation to the stream of its
first use.)

The arithmetic runs in the CUDA kernels; sums are FP32 in a fixed order.
"""
from __future__ import annotations

import torch

from . import nvfp4 as F


def on_stream(stream):
    """Context in which torch allocates for `stream` (a torch stream or a raw
    handle), so that memory freed on return is reused in that stream's order."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def empty(shape, dtype, device, stream=None):
    """torch.empty in the order of `stream` (None: the current one)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with on_stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def rows_of(t, name, stream=None):
    """t as rows whose elements are neighbours (a copy only where they are not)."""
    if t.dim() != 2:
        raise ValueError(f"{name}: expected rows [n, D], got shape {tuple(t.shape)}")
    n, D = t.shape
    if D == 0:
        raise ValueError(f"{name}: rows of width 0")
    ld, step = t.stride()
    if (D > 1 and step != 1) or (n > 1 and ld < D):
        if stream is None:
            return t.contiguous()
        with on_stream(stream):
            return t.contiguous()
    return t


def check_routes(route_pos, expert_offsets=None):
    if route_pos.dim() != 2 or route_pos.dtype != torch.int32 or not route_pos.is_contiguous():
        raise ValueError("route_pos: expected contiguous int32 [T, topk]")
    if expert_offsets is not None and (expert_offsets.dim() != 1 or expert_offsets.numel() < 2
                                       or expert_offsets.dtype != torch.int32
                                       or not expert_offsets.is_contiguous()):
        raise ValueError("expert_offsets: expected contiguous int32 [E + 1]")


def _weights(weights, route_pos, stream=None):
    if weights.shape != route_pos.shape or weights.dtype != torch.float32:
        raise ValueError("weights: expected FP32 of route_pos' shape")
    if stream is None or weights.is_contiguous():
        return weights.contiguous()
    with on_stream(stream):
        return weights.contiguous()


def _dispatch(x, route_pos, expert_offsets, R, stream=None):
    out = empty((R, x.shape[1]), x.dtype, x.device, stream)
    F.nvfp4_tokens_dispatch(x, route_pos, expert_offsets, out, stream)
    return out


def _combine(y, route_pos, weights, stream=None):
    out = empty((route_pos.shape[0], y.shape[1]), y.dtype, y.device, stream)
    F.nvfp4_tokens_combine(y, route_pos, weights, out, stream)
    return out


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, route_pos, expert_offsets, R):
        ctx.save_for_backward(route_pos)
        return _dispatch(x, route_pos, expert_offsets, R)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        return dispatch_grad(dout, *ctx.saved_tensors), None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, route_pos, weights, expert_offsets):
        ctx.offsets = expert_offsets is not None
        ctx.save_for_backward(y, route_pos, weights,
                              *([expert_offsets] if ctx.offsets else []))
        return _combine(y, route_pos, weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        y, route_pos, weights, *rest = ctx.saved_tensors
        dy, dw = combine_grad(dout, y, route_pos, weights, rest[0] if rest else None)
        return dy, None, dw, None


def dispatch(x, route_pos, expert_offsets=None, R=None, stream=None):
    """x [T, D] -> rows in expert order [R, D] (R: T * topk unless given).  Rows
    past expert_offsets[E] are zero; without expert_offsets, rows that no route
    names are left unwritten."""
    check_routes(route_pos, expert_offsets)
    x = rows_of(x, "x", stream)
    if x.shape[0] != route_pos.shape[0]:
        raise ValueError(f"{x.shape[0]} rows for the routes of {route_pos.shape[0]} tokens")
    R = route_pos.numel() if R is None else R
    if stream is None and x.requires_grad and torch.is_grad_enabled():
        return _Dispatch.apply(x, route_pos, expert_offsets, R)
    return _dispatch(x, route_pos, expert_offsets, R, stream)


def dispatch_grad(dout, route_pos, stream=None):
    """Gradient of `dispatch`: dout [R, D] -> [T, D], the sum over each token's
    routes."""
    check_routes(route_pos)
    return _combine(rows_of(dout, "dout", stream), route_pos, None, stream)


def combine(y, route_pos, weights=None, expert_offsets=None, stream=None):
    """y [R, D] in expert order -> [T, D]: the sum of each token's routes, times
    weights (FP32 [T, topk]) where given.  expert_offsets is used by the
    backward pass alone: the gradient's rows past expert_offsets[E] are zero."""
    check_routes(route_pos, expert_offsets)
    y = rows_of(y, "y", stream)
    if weights is not None:
        weights = _weights(weights, route_pos, stream)
    if stream is None and torch.is_grad_enabled() and (
            y.requires_grad or (weights is not None and weights.requires_grad)):
        if weights is None:
            weights = torch.ones(route_pos.shape, dtype=torch.float32, device=y.device)
        return _Combine.apply(y, route_pos, weights, expert_offsets)
    return _combine(y, route_pos, weights, stream)


def combine_grad(dout, y, route_pos, weights, expert_offsets=None, stream=None):
    """Gradient of `combine`: (dy [R, D], dweights FP32 [T, topk]).  Rows of dy
    past expert_offsets[E] are zero; without expert_offsets, rows that no route
    names are left unwritten."""
    check_routes(route_pos, expert_offsets)
    weights = _weights(weights, route_pos, stream)
    dout, y = rows_of(dout, "dout", stream), rows_of(y, "y", stream)
    if dout.shape != (route_pos.shape[0], y.shape[1]) or dout.dtype != y.dtype:
        raise ValueError("dout: expected [T, D] of y's width and type")
    dy = empty(y.shape, y.dtype, y.device, stream)
    dw = empty(route_pos.shape, torch.float32, y.device, stream)
    F.nvfp4_tokens_combine_grad(dout, y, route_pos, weights, expert_offsets, dy, dw, stream)
    return dy, dw
