"""Root-mean-square norm of rows, with the residual's addition and its gradient,
and with 8-bit output for the FP8 products.

    h = x + residual                          (rounded to the rows' type)
    y = h / sqrt(mean(h^2) + eps) * weight    (FP32, rounded once)

Rows [.., D] are BF16, FP16 or FP32 of any width up to 16384; the weight [D] has the
rows' type or is FP32.  Rows whose elements are not neighbours, or whose stride differs
from a dense matrix's by no multiple of 16 bytes, are copied first.  The squares are FP32:
rows whose sum of squares passes its range (elements from about 2^57 in the widest rows, 2^63
in narrow ones) have rstd 0, squares below it (elements under 2^-63, which only tells where
eps is as small) lose bits, and a row of zeros without an eps is 0 / 0.

`rms_norm` takes part in autograd; `rms_norm_grad` is its gradient as a plain call, which
enqueues kernels only (the one for a captured step: autograd's own bookkeeping can use other
streams).  `rms_norm_fp8` gives E4M3 codes and one FP32 scale per 128 columns, as
fp8.quantize_rows does, from the unrounded y: it rounds and has no derivative.  There is no
forward-mode derivative.

Work goes to the current stream of the tensors' device, whichever device is current,
or to `stream` (a torch stream of that device or a raw handle).
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from .nvfp4 import native
from .tokens import on_stream, refuse_tangents


def _rows(t):
    return t if t is None or t.dim() == 2 else t.reshape(-1, t.shape[-1])


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        out = native().rms_norm(x, weight, residual, eps, False)
        ctx.eps = eps
        ctx.save_for_backward(x if residual is None else out[1], weight)
        ctx.set_materialize_grads(False)
        return out[0] if residual is None else out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        if dy is None:                        # only the sum was used
            return dh, None, dh if ctx.needs_input_grad[2] else None, None
        dx, dweight = native().rms_norm_grad(dy, h, weight, dh, ctx.eps)
        return (dx if ctx.needs_input_grad[0] else None,
                dweight if ctx.needs_input_grad[1] else None,
                dx if ctx.needs_input_grad[2] else None, None)


def rms_norm(x, weight, residual=None, eps: float = 1e-6, stream=None):
    """x [.., D] -> y, or, with a residual of x's shape, (y, h)."""
    if forward_ad._current_level >= 0:
        refuse_tangents(x, weight, residual)
    if stream is not None:
        with on_stream(stream, x.device):
            return rms_norm(x, weight, residual, eps)
    if x.dim() != 2:
        if x.dim() == 0 or (residual is not None and residual.shape != x.shape):
            raise ValueError("x: expected rows [.., D], residual: of x's shape")
        out = rms_norm(_rows(x), weight, _rows(residual), eps)
        return out.view(x.shape) if residual is None else tuple(t.view(x.shape) for t in out)
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad or (
            residual is not None and residual.requires_grad)):
        return _RmsNorm.apply(x, weight, residual, eps)
    out = native().rms_norm(x, weight, residual, eps, False)
    return out[0] if residual is None else out


def rms_norm_grad(dy, h, weight, dh=None, eps: float = 1e-6, stream=None):
    """Gradient of `rms_norm` at h (x itself without a residual): (dx, dweight).  dx is
    the gradient of x and of the residual alike; dh is that of h as an output of its
    own."""
    if forward_ad._current_level >= 0:
        refuse_tangents(dy, h, weight, dh)
    if stream is not None:
        with on_stream(stream, h.device):
            return rms_norm_grad(dy, h, weight, dh, eps)
    if h.dim() != 2:
        if h.dim() == 0 or dy.shape != h.shape or (dh is not None and dh.shape != h.shape):
            raise ValueError("h: expected rows [.., D], dy and dh: of h's shape")
        dx, dweight = native().rms_norm_grad(_rows(dy), _rows(h), weight, _rows(dh), eps)
        return dx.view(h.shape), dweight
    return native().rms_norm_grad(dy, h, weight, dh, eps)


def rms_norm_fp8(x, weight, residual=None, eps: float = 1e-6, stream=None):
    """x [T, D] (BF16 or FP16, D % 16 == 0) -> (codes float8_e4m3fn [T, D], scales FP32
    [ceil(D / 128), T]), with a residual (codes, scales, h): the operands of
    fp8.linear_codes."""
    if forward_ad._current_level >= 0:
        refuse_tangents(x, weight, residual)
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad or (
            residual is not None and residual.requires_grad)):
        raise RuntimeError("rms_norm_fp8 rounds and has no derivative: use rms_norm, or no_grad")
    if stream is not None:
        with on_stream(stream, x.device):
            return native().rms_norm(x, weight, residual, eps, True)
    return native().rms_norm(x, weight, residual, eps, True)
