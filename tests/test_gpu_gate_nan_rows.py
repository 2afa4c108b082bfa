"""A NaN among logits that are -infinities otherwise: the softmax has no value at all there, as where
other logits are finite.  With a bias all sums are then NaN, and the lowest numbers are chosen."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import gating

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [4, 40, 100, 300])
def test_nan_among_infinities(E):
    l = torch.full((3, E), -float("inf"), device="cuda")
    l[0, E - 1] = float("nan")
    l[1, E - 1] = float("nan")
    l[1, 1] = 0.5                            # row 2: nothing but -infinities
    bias = torch.linspace(0, 1, E, device="cuda")
    for renormalize in (True, False):
        ids, w = gating.topk_gate(l, 3, bias, "softmax", renormalize)
        assert ids.tolist() == [[0, 1, 2], [0, 1, 2], [E - 1, E - 2, E - 3]]
        assert bool(torch.isnan(w[:2]).all()) and bool((w[2] == 0).all())
        ids, w = gating.topk_gate(l, 3, None, "softmax", renormalize)
        assert ids.tolist() == [[E - 1, 0, 1], [E - 1, 1, 0], [0, 1, 2]]
        assert bool(torch.isnan(w[:2]).all()) and bool((w[2] == 0).all())
