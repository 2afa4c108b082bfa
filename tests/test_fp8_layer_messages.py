"""What step_few says where it does not take a call (no GPU needed: the library's answer is
played)."""
import types

import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import moe
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F


def rows(T, K=64):
    return torch.zeros((T, K), dtype=torch.bfloat16)


def test_reasons(monkeypatch):
    monkeypatch.setattr(F, "native", lambda: types.SimpleNamespace(moe_layer=lambda *a: None))
    codes = torch.zeros((2, 128, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    down = torch.zeros((2, 64, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros((2, 1, 1))
    mlp = moe.Fp8MLP((codes, scales), (down, scales))

    def call(T, topk):
        return mlp.step_few(rows(T), torch.zeros((T, topk), dtype=torch.int32), torch.zeros((T, topk)))

    with pytest.raises(ValueError, match="at most 8 tokens"):
        call(9, 2)
    with pytest.raises(ValueError, match="multiples of 16") as e:
        call(8, 3)
    assert "at most 8 tokens" not in str(e.value) and "step()" in str(e.value)
    assert call(0, 2).shape == (0, 64)
