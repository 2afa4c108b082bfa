"""Routing that moe.Fp8MLP refuses: other types or layouts of the experts' numbers
would be read as if they were dense 32-bit ones (no GPU needed)."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import moe


def test_expert_numbers_of_other_types_and_layouts():
    def codes(*shape):
        return torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn)

    layer = moe.Fp8MLP((codes(4, 256, 64), torch.zeros(4, 2, 1)),
                       (codes(4, 64, 128), torch.zeros(4, 1, 1)))
    ids = torch.zeros((8, 2), dtype=torch.int32)
    x, weights = torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((8, 2))
    for bad in (ids.long(), ids.float(), ids[:, 0], ids.t(), ids[:, :1]):
        with pytest.raises(ValueError, match="topk_ids"):
            layer.route(bad)
        with pytest.raises(ValueError, match="topk_ids"):
            layer.step(x, bad, weights)
    with pytest.raises(ValueError, match="CUDA"):     # the right type: on to the device's check
        layer.route(ids)
