"""No token at all, as a batch may have it between requests or an expert-parallel rank
in a step: results of no rows, or zeros where the buffer has rows."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8, moe
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F
from test_gpu_fp8 import weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("topk", [1, 2, 8])
@pytest.mark.parametrize("silu_mul", [False, True])
def test_expert_linear_and_quantiser(topk, silu_mul):
    E, N, K = 8, 256, 128
    w, ws = weights(1, E, N, K)
    x = torch.empty((0, 2 * K if silu_mul else K), dtype=torch.bfloat16, device="cuda")
    pos = torch.empty((0, topk), dtype=torch.int32, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    assert fp8.expert_linear(x, w, ws, off, pos, silu_mul=silu_mul).shape == (0, N)
    assert fp8.expert_linear(x, w, ws, off, silu_mul=silu_mul).shape == (0, N)
    for R in (3, 200):
        y = fp8.expert_linear(x, w, ws, off, pos, R, silu_mul)
        assert torch.equal(y, torch.zeros((R, N), dtype=torch.bfloat16, device="cuda"))
    codes, scales = fp8.quantize_rows(x, pos, silu_mul=silu_mul)
    assert codes.shape == (0, K) and scales.shape == (1, 0)
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_layer():
    layer = moe.Fp8MLP(weights(1, 4, 256, 128), weights(2, 4, 64, 128))
    out = layer.step(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"),
                     torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                     torch.empty((0, 2), device="cuda"))
    assert out.shape == (0, 64) and out.dtype == torch.bfloat16
    assert F.nvfp4_device_status() == F.NVFP4_OK
