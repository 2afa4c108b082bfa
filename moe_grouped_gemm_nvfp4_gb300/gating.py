"""Top-k gate of an MoE layer: from the router's logits to the chosen experts and
their weights, and the gradient.

Scores are softmax(logits) or sigmoid(logits).  Chosen are the topk largest logits or,
with a bias, the topk largest score + bias: best first, the lower number first among
equals, a NaN as the largest value.  The weights are the chosen scores (without the
bias), divided by their sum with renormalize, times scale.  Renormalised weights are ratios and
hold also where the scores are below FP32's range.  A row of -infinities has softmax scores
0, and renormalised weights 0 where all chosen logits are -infinities.  Sums that FP32
rounding could swap are compared in FP64.

`topk_gate` takes part in autograd (the gradient of the logits; the choice and the bias
have none); `topk_gate_grad` is the gradient as a plain call, which enqueues kernels
only (the one for a captured step).  Logits are BF16, FP16 or FP32 [T, E] of any row stride, at most 1024 experts and
32 chosen ones.  There is no forward-mode derivative.

Work goes to the current stream of the tensors' device, whichever device is current,
or to `stream` (a torch stream of that device or a raw handle).
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from .nvfp4 import native
from .tokens import on_stream, refuse_tangents

SCORES = ("softmax", "sigmoid")


def is_sigmoid(score: str) -> bool:
    if score not in SCORES:
        raise ValueError(f"score: expected one of {SCORES}, got {score!r}")
    return score == "sigmoid"


class _TopkGate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, bias, sigmoid, renormalize, scale):
        ids, weights = native().topk_gate(logits, topk, bias, sigmoid, renormalize, scale)
        ctx.save_for_backward(logits, ids)
        ctx.rule = (sigmoid, renormalize, scale)
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, dweights):
        logits, ids = ctx.saved_tensors
        return native().topk_gate_grad(dweights, logits, ids, *ctx.rule), *([None] * 5)


def topk_gate(logits, topk: int, bias=None, score: str = "softmax", renormalize: bool = True,
              scale: float = 1.0, stream=None):
    """Logits [T, E] -> (ids int32 [T, topk], weights FP32 [T, topk])."""
    if forward_ad._current_level >= 0:
        refuse_tangents(logits, bias)
    sigmoid = is_sigmoid(score)
    if stream is not None:
        with on_stream(stream, logits.device):
            return topk_gate(logits, topk, bias, score, renormalize, scale)
    if logits.requires_grad and torch.is_grad_enabled():
        return _TopkGate.apply(logits, topk, bias, sigmoid, renormalize, scale)
    return native().topk_gate(logits, topk, bias, sigmoid, renormalize, scale)


def topk_gate_grad(dweights, logits, topk_ids, score: str = "softmax", renormalize: bool = True,
                   scale: float = 1.0, stream=None):
    """Gradient of the weights of `topk_gate` (dweights FP32 [T, topk], topk_ids its
    choice) -> dlogits [T, E] of the logits' type."""
    if forward_ad._current_level >= 0:
        refuse_tangents(dweights, logits)
    sigmoid = is_sigmoid(score)
    if stream is not None:
        with on_stream(stream, logits.device):
            return topk_gate_grad(dweights, logits, topk_ids, score, renormalize, scale)
    return native().topk_gate_grad(dweights, logits, topk_ids, sigmoid, renormalize, scale)
