"""Equal logits under equal biases are equal sums, wherever their experts lie in the warp: the
lower number first."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import gating

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [20, 52, 100, 128, 200, 300, 600, 1024])
def test_equal_sums(E, score):
    g = torch.Generator().manual_seed(E)
    # few values: many equals in a row
    l = (torch.randn((1000, E), generator=g) + 10).bfloat16().cuda()
    masked = torch.where(torch.rand(E, generator=g) < 0.5, -float("inf"), 0.01)
    for bias in (masked, torch.full((E,), 0.01), torch.full((E,), -0.3), torch.zeros(E)):
        bias = bias.cuda()
        s = torch.softmax(l.double(), 1) if score == "softmax" else 1 / (1 + torch.exp(-l.double()))
        for topk in (1, 8, min(E, 30)):
            ids, _ = gating.topk_gate(l, topk, bias, score)
            want = torch.sort(s + bias.double(), dim=1, descending=True, stable=True).indices[:, :topk]
            assert torch.equal(ids.long(), want)
