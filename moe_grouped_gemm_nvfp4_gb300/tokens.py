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

import contextlib

import torch

from . import nvfp4 as F


def on_stream(stream):
    """Context in which torch allocates for `stream` (a torch stream or a raw
    handle; None: the current one), so that memory freed on return is reused in
    that stream's order."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def rows_of(t, name):
    """t as rows whose elements are neighbours (a copy only where they are not)."""
    if t.dim() != 2:
        raise ValueError(f"{name}: expected rows [n, D], got shape {tuple(t.shape)}")
    if t.shape[1] == 0:
        raise ValueError(f"{name}: rows of width 0")
    n, D = t.shape
    if (D > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < D):
        return t.contiguous()
    return t


def check_routes(route_pos, expert_offsets=None):
    if route_pos.dim() != 2 or route_pos.dtype != torch.int32 or not route_pos.is_contiguous():
        raise ValueError("route_pos: expected contiguous int32 [T, topk]")
    if expert_offsets is not None and (expert_offsets.dim() != 1 or expert_offsets.numel() < 2
                                       or expert_offsets.dtype != torch.int32
                                       or not expert_offsets.is_contiguous()):
        raise ValueError("expert_offsets: expected contiguous int32 [E + 1]")


def _check_weights(weights, route_pos):
    if weights.shape != route_pos.shape or weights.dtype != torch.float32:
        raise ValueError("weights: expected FP32 of route_pos' shape")


def _dispatch(x, route_pos, expert_offsets, R, stream=None):
    with on_stream(stream):
        out = torch.empty((R, x.shape[1]), dtype=x.dtype, device=x.device)
    F.nvfp4_tokens_dispatch(x, route_pos, expert_offsets, out, stream)
    return out


def _combine(y, route_pos, weights, stream=None):
    with on_stream(stream):
        out = torch.empty((route_pos.shape[0], y.shape[1]), dtype=y.dtype, device=y.device)
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
    x = rows_of(x, "x")
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
    return _combine(rows_of(dout, "dout"), route_pos, None, stream)


def combine(y, route_pos, weights=None, expert_offsets=None, stream=None):
    """y [R, D] in expert order -> [T, D]: the sum of each token's routes, times
    weights (FP32 [T, topk]) where given.  expert_offsets is used by the
    backward pass alone: the gradient's rows past expert_offsets[E] are zero."""
    check_routes(route_pos, expert_offsets)
    y = rows_of(y, "y")
    if weights is not None:
        _check_weights(weights, route_pos)
        weights = weights.contiguous()
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
    _check_weights(weights, route_pos)
    dout, y = rows_of(dout, "dout"), rows_of(y, "y")
    if dout.shape != (route_pos.shape[0], y.shape[1]) or dout.dtype != y.dtype:
        raise ValueError("dout: expected [T, D] of y's width and type")
    with on_stream(stream):
        weights = weights.contiguous()
        dy = torch.empty(y.shape, dtype=y.dtype, device=y.device)
        dw = torch.empty(route_pos.shape, dtype=torch.float32, device=y.device)
    F.nvfp4_tokens_combine_grad(dout, y, route_pos, weights, expert_offsets, dy, dw, stream)
    return dy, dw
