"""FP8 products of activations near the largest finite BF16 values, whose results
are finite: few rows (one launch on the CUDA cores) and more (tensor cores) agree
with 64-bit arithmetic alike.  Bounds as in test_gpu_fp8."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F
from test_gpu_fp8 import check, check_experts, oracle_rows, product
from test_gpu_tokens import normal, routes

pytestmark = pytest.mark.gpu

LARGEST = float(torch.finfo(torch.bfloat16).max)


def weights(seed, E, N, K, sigma):
    return fp8.quantize_weights(normal(seed, (E, N, K), torch.float32) * sigma)


def large(M, K, value):
    """Rows of one magnitude, random signs, one of them with zeros in between."""
    x = torch.where(normal(M + K, (M, K), torch.float32) > 0, value, -value)
    x[M // 2, ::3] = 0
    return x.to(torch.bfloat16)


# sums of up to K = 2048 products of value * sigma stay finite
@pytest.mark.parametrize("value,sigma", [(5e34, 0.02), (8e35, 0.02), (4e36, 0.02), (LARGEST, 1e-5)])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 40])
@pytest.mark.parametrize("N,K", [(256, 512), (130, 2048), (640, 144)])
def test_rows_of_large_activations(M, N, K, value, sigma):
    w, ws = weights(N + K, 1, N, K, sigma)
    x = large(M, K, value)
    ref, mag = product(*oracle_rows(x), w[0], ws[0])
    assert mag.max() < 2.0 ** 127
    check(fp8.linear(x, w[0], ws[0]), ref, mag, K)


@pytest.mark.parametrize("T,topk", [(2, 2), (4, 4), (40, 4)])
@pytest.mark.parametrize("gather", [True, False])
def test_routes_of_large_activations(T, topk, gather):
    E, N, K = 8, 256, 512
    w, ws = weights(3, E, N, K, 0.02)
    pos, off = routes(T, T, topk, E)
    x = large(T if gather else T * topk, K, 4e36)
    y = fp8.expert_linear(x, w, ws, off, pos if gather else None)
    check_experts(x, w, ws, pos, off, T * topk, gather, y)
    assert F.nvfp4_device_status() == F.NVFP4_OK


@pytest.mark.parametrize("R", [4, 40])
def test_gated_halves_of_large_activations(R):
    """SiLU(gate) * up = 64 * 5e34 in every place of the sum, up to the sign."""
    E, N, K = 1, 128, 256
    w, ws = weights(5, E, N, K, 0.02)
    gu = torch.cat([torch.full((R, K), 64.0, dtype=torch.bfloat16, device="cuda"),
                    large(R, K, 5e34)], dim=1)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    y = fp8.expert_linear(gu, w, ws, off, silu_mul=True)
    codes, scales = fp8.quantize_rows(gu, silu_mul=True)
    ref, mag = product(codes, scales, w[0], ws[0])
    check(y, ref, mag, K)


@pytest.mark.parametrize("M", [2, 4])
@pytest.mark.parametrize("N,K", [(256, 512), (130, 2064)])
def test_few_rows_with_nan_or_infinity_stay_alone(M, N, K):
    w, ws = weights(1, 1, N, K, 0.02)
    x = normal(0, (M, K), torch.bfloat16)
    want = fp8.linear(x, w[0], ws[0])
    for bad in (float("inf"), float("nan")):
        z = x.clone()
        z[1, K - 1] = bad
        y = fp8.linear(z, w[0], ws[0])
        assert torch.isnan(y[1]).all()
        keep = [m for m in range(M) if m != 1]
        assert torch.equal(y[keep], want[keep])
