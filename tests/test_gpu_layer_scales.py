"""The MoE layer for a few tokens with scales far from one, in range: the experts' products, h
and its scales in numbers whose exponents the tests elsewhere do not reach.

Tolerance as in test_gpu_moe_layer.py.
"""
import pytest
import torch

from test_gpu_moe_layer import experts64, rel, small, tolerance

from moe_grouped_gemm_nvfp4_gb300 import moe
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

pytestmark = pytest.mark.gpu


def check(mlp, x, ids, weights):
    out = mlp.step_few(x, ids, weights)
    ref = experts64(x, ids, weights, mlp.gate_up, mlp.down)
    top = float(ref.abs().max())
    assert 1e-37 < top < 3e38               # nothing drops out of the comparison
    assert rel(out, ref) <= tolerance(x.dtype)
    assert F.nvfp4_device_status() == F.NVFP4_OK


@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("exponent,back", [(50, 0), (-40, 0), (100, -100), (-90, 90), (90, -110),
                                           (30, -60), (-100, 70)])
def test_rows_and_weights_far_from_one(exponent, back, T):
    """x times 2^exponent, gate_up times 2^back; h is the square of their sum, and keeps in
    range with its scale (the least is 2^-100 / 448)."""
    g, mlp, x = small(7)
    weights = torch.rand((6, 3), generator=g).cuda()
    ids = torch.rand((6, 8), generator=g).topk(3, dim=1).indices.to(torch.int32).cuda()
    codes, scales = mlp.gate_up
    far = moe.Fp8MLP((codes, (scales.double() * 2.0 ** back).float()), mlp.down)
    rows = (x.double() * 2.0 ** exponent).to(torch.bfloat16)
    check(far, rows[:T], ids[:T], weights[:T])


@pytest.mark.parametrize("exponent", [100, -90])
def test_routing_and_down_weights_far_from_one(exponent):
    g, mlp, x = small(8)
    weights = torch.rand((6, 3), generator=g).cuda()
    ids = torch.rand((6, 8), generator=g).topk(3, dim=1).indices.to(torch.int32).cuda()
    codes, scales = mlp.down
    far = moe.Fp8MLP(mlp.gate_up, (codes, (scales.double() * 2.0 ** exponent).float()))
    check(far, x, ids, weights)
    check(far, x, ids, weights * 2.0 ** -(exponent // 2))
