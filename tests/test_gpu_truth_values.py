"""Arguments that are neither true nor false are refused like other arguments."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8, gating

pytestmark = pytest.mark.gpu


def test_truth_values():
    both = torch.tensor([True, False])
    l = torch.randn((4, 8), device="cuda")
    ids, w = gating.topk_gate(l, 2)
    codes, scales = fp8.quantize_weights(torch.randn((2, 64, 32), device="cuda"))
    x = torch.randn((4, 64), device="cuda").bfloat16()
    offsets = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: gating.topk_gate(l, 2, renormalize=both),
                 lambda: gating.topk_gate_grad(w, l, ids, renormalize=both),
                 lambda: fp8.expert_linear(x, codes, scales, offsets, silu_mul=both)):
        with pytest.raises(ValueError, match="true or false"):
            call()
    assert torch.equal(gating.topk_gate(l, 2, renormalize=1)[0], ids)
