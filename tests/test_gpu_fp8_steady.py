"""FP8 products whose CTAs take several units of many K blocks: every stage and
accumulator of the rings goes round more than once, and the factors' groups of four
K blocks end in whole and partial ones before the next unit's, for each tile width and
both ways of storing rows.  Bounds as in test_gpu_fp8 (64-bit sums over the same codes
and scales)."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F
from test_gpu_fp8 import check, check_experts, product, weights
from test_gpu_tokens import normal, routes

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# rows of 16, 32, 64 and 128 a tile; outputs in whole 16-byte chunks and in odd rows
@pytest.mark.parametrize("M,N", [(16, 60000), (16, 59999), (30, 60000), (30, 59997), (70, 30000),
                                 (70, 30001), (5000, 2048), (5000, 2047)])
@pytest.mark.parametrize("K", [528, 656, 1040, 1168])
def test_dense(M, N, K):
    tile = 16 if M <= 16 else 32 if M <= 32 else 64 if M <= 80 else 128
    assert -(-M // tile) * -(-N // 128) > 2 * sms()
    w, ws = weights(N + K, 1, N, K)
    x = normal(M, (M, K), torch.bfloat16)
    y = fp8.linear(x, w[0], ws[0])
    codes, scales = fp8.quantize_rows(x)
    ref, mag = product(codes, scales, w[0], ws[0])
    check(y, ref, mag, K)
    assert torch.equal(fp8.linear(x, w[0], ws[0]), y)
    assert F.nvfp4_device_status() == F.NVFP4_OK


# routes per expert that give tiles of 16, 32, 64 and 128
@pytest.mark.parametrize("per_expert", [4, 12, 40, 150])
@pytest.mark.parametrize("N", [1024, 1021])
@pytest.mark.parametrize("K", [656, 1168])
@pytest.mark.parametrize("gather", [True, False])
def test_grouped(per_expert, N, K, gather):
    E, topk = 64, 4
    T = E * per_expert // topk
    assert E * -(-N // 128) > 2 * sms()
    w, ws = weights(N + K, E, N, K)
    pos, off = routes(T + N, T, topk, E, 0.1)
    x = normal(K, (T if gather else T * topk, K), torch.float16 if gather else torch.bfloat16)
    y = fp8.expert_linear(x, w, ws, off, pos if gather else None)
    check_experts(x, w, ws, pos, off, T * topk, gather, y)
    assert F.nvfp4_device_status() == F.NVFP4_OK


@pytest.mark.parametrize("T,topk,E,N,K", [(30, 4, 8, 130, 272), (500, 4, 8, 1000, 656),
                                          (64, 4, 64, 1024, 1168), (2400, 4, 64, 1021, 656)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pad", [0, 5, 8])
def test_grouped_gemm_of_codes(T, topk, E, N, K, dtype, pad):
    """The product alone: output types, row strides, and zeros past the live rows."""
    w, ws = weights(N + K, E, N, K)
    pos, off = routes(T, T, topk, E, 0.25)
    R, live = T * topk, int(off[-1])
    codes, scales = fp8.quantize_rows(normal(K, (T, K), torch.bfloat16), pos)
    wide = torch.full((R, N + pad), float("nan"), dtype=dtype, device="cuda")
    F.nvfp4_fp8_grouped_gemm(codes, scales, w, ws, off, wide[:, :N])
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            ref, mag = product(codes[a:b], scales[:, a:b], w[e], ws[e])
            check(wide[a:b, :N], ref, mag, K, f"expert {e}")
    assert live < R and not wide[live:, :N].any()
    assert int(torch.isnan(wide).sum()) == R * pad               # nothing else written
    assert F.nvfp4_device_status() == F.NVFP4_OK
