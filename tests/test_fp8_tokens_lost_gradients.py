"""Calls that would return a result without the derivative that was asked for
raise instead (no GPU needed: they refuse before any device call)."""
import pytest
import torch
from torch.autograd import forward_ad

from moe_grouped_gemm_nvfp4_gb300 import fp8, tokens


def operands():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    codes = torch.zeros((2, 128, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    return x, codes, torch.zeros((2, 1, 1)), torch.zeros(3, dtype=torch.int32)


@pytest.mark.parametrize("which", ["x", "w", "w_scale"])
def test_products_refuse_every_operand_that_requires_a_gradient(which):
    x, codes, scales, off = operands()
    named = {"x": x, "w": codes, "w_scale": scales}
    named[which] = torch.nn.Parameter(named[which])
    with pytest.raises(RuntimeError, match="not differentiable"):
        fp8.expert_linear(named["x"], named["w"], named["w_scale"], off)
    dense = {**named, "w": named["w"][0], "w_scale": named["w_scale"][0]}
    with pytest.raises(RuntimeError, match="not differentiable"):
        fp8.linear(**dense)
    # frozen parameters, and parameters under no_grad, go on to the device's checks
    with torch.no_grad(), pytest.raises(ValueError):
        fp8.linear(**dense)
    named[which].requires_grad_(False)
    with pytest.raises(ValueError):
        fp8.expert_linear(named["x"], named["w"], named["w_scale"], off)


def test_missing_operands_stay_argument_errors():
    x, codes, scales, off = operands()
    with pytest.raises(ValueError):
        fp8.linear(x, codes[0], None)
    with pytest.raises(ValueError):
        fp8.expert_linear(x, None, scales, off)


def test_tangents_are_refused():
    x, codes, scales, off = operands()
    pos = torch.zeros((4, 2), dtype=torch.int32)
    y, w = torch.zeros((8, 64)), torch.zeros((4, 2))
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))

        calls = [lambda: tokens.dispatch(dual(x), pos, off),
                 lambda: tokens.dispatch_grad(dual(y), pos),
                 lambda: tokens.combine(dual(y), pos, w),
                 lambda: tokens.combine(y, pos, dual(w)),
                 lambda: tokens.combine_grad(dual(x.float()), y, pos, w),
                 lambda: tokens.combine_grad(x.float(), dual(y), pos, w),
                 lambda: tokens.combine_grad(x.float(), y, pos, dual(w)),
                 lambda: fp8.linear(dual(x), codes[0], scales[0]),
                 lambda: fp8.linear(x, codes[0], dual(scales[0])),
                 lambda: fp8.expert_linear(dual(x), codes, scales, off)]
        for call in calls:
            with pytest.raises(RuntimeError, match="tangent"):
                call()
            with torch.no_grad(), pytest.raises(RuntimeError, match="tangent"):
                call()
        with pytest.raises(ValueError):            # no tangent: on to the device's checks
            tokens.dispatch(x, pos, off)
        with pytest.raises(ValueError):
            tokens.combine(y, pos)
