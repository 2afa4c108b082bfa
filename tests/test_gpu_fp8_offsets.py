"""Offsets that go back and forth: reported, every element of the output from one of
the experts that claim it (or zero, since expert_offsets[E] = 0 says that no row is
live), and the next call right again."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F
from test_gpu_tokens import normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,E,N", [(600, 8, 256), (40, 8, 130), (9000, 40, 512), (9000, 40, 333)])
def test_overlapping_experts(R, E, N):
    K = 656
    w, ws = fp8.quantize_weights(normal(N, (E, N, K), torch.float32) * 0.02)
    x = normal(1, (R, K), torch.bfloat16)
    bad = torch.tensor([0 if e % 2 == 0 else R for e in range(E + 1)], dtype=torch.int32).cuda()
    y = fp8.expert_linear(x, w, ws, bad)
    assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK
    one = y == 0
    for e in range(0, E, 2):
        only = torch.tensor([0] * (e + 1) + [R] * (E - e), dtype=torch.int32).cuda()
        one |= y == fp8.expert_linear(x, w, ws, only)
    assert one.all()
    assert F.nvfp4_device_status() == F.NVFP4_OK
