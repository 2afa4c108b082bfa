"""Gradient of the gate where one expert has almost all of the score: its own gradient is
p (1 - p) dp, which differences of values near p dp do not hold.

Reference: dl_j = p_j sum_i p_i (dp_j - dp_i) in 64 bits (over all experts, or over the chosen
with renormalised weights).  Tolerance: relative to the sum of the terms' magnitudes, each with
the rounding of its factors: (|l - max| + 32) * 2^-24 for a score, twice (two scores a term),
and the sums' own, below E + 8 additions of 2^-24.
"""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import gating

pytestmark = pytest.mark.gpu


def check(dl, l, ids, g64, p, dp, slope=1.0):
    pair = (dp[:, :, None] - dp[:, None, :]) * p[:, None, :] * p[:, :, None] * slope
    ref, size = pair.sum(2), pair.abs().sum(2)
    far = float((l.max() - l.min()).clamp(max=90))
    unit = (2 * (far + 32) + p.shape[1] + 8) * 2.0 ** -24
    # (the shift by the largest's own gradient can triple the terms)
    assert bool(((dl.double() - ref).abs()
                 <= ref.abs() * torch.finfo(dl.dtype).eps / 2 + 3 * unit * size + 2.0 ** -148).all())
    assert bool((ref != 0).any())


def saturated(g, T, E, gap):
    l = torch.randn((T, E), generator=g)
    top = torch.randint(0, E, (T, 1), generator=g)
    return l.scatter(1, top, (4 + gap + torch.rand((T, 1), generator=g))).cuda()


@pytest.mark.parametrize("gap", [4.0, 12.0, 16.0, 20.0, 40.0])
@pytest.mark.parametrize("E,topk", [(2, 1), (16, 2), (60, 6), (128, 8), (300, 8), (700, 1)])
def test_softmax(E, topk, gap):
    g = torch.Generator().manual_seed(E)
    l = saturated(g, 40, E, gap)
    ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :topk].int()
    dw = torch.randn((40, topk), generator=g).cuda()
    dl = gating.topk_gate_grad(dw, l, ids, "softmax", False, 1.5)
    p = torch.softmax(l.double(), 1)
    dp = torch.zeros_like(p).scatter(1, ids.long(), 1.5 * dw.double())
    check(dl, l, ids, None, p, dp)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gap", [4.0, 12.0, 16.0, 20.0, 40.0])
@pytest.mark.parametrize("E,topk", [(2, 2), (16, 2), (60, 6), (128, 8), (300, 32)])
def test_renormalised(E, topk, gap, score):
    g = torch.Generator().manual_seed(E)
    l = saturated(g, 40, E, gap)
    if score == "sigmoid":
        l -= 44 + gap                       # (scores that follow the exponential)
    ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :topk].int()
    dw = torch.randn((40, topk), generator=g).cuda()
    dl = gating.topk_gate_grad(dw, l, ids, score, True, 1.5)
    chosen = l.double().gather(1, ids.long())
    logs = chosen if score == "softmax" else torch.nn.functional.logsigmoid(chosen)
    slope = 1.0 if score == "softmax" else torch.sigmoid(-chosen)[:, :, None]
    check(dl.gather(1, ids.long()), l, ids, None, torch.softmax(logs, 1), 1.5 * dw.double(), slope)


def test_a_dominant_expert_that_is_not_chosen():
    """Where the caller's choice leaves the largest out, and where an expert is named twice."""
    g = torch.Generator().manual_seed(5)
    l = saturated(g, 40, 30, 16.0)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    dw = torch.randn((40, 3), generator=g).cuda()
    p = torch.softmax(l.double(), 1)
    for ids in (order[:, 1:4], order[:, [0, 0, 2]]):
        dl = gating.topk_gate_grad(dw, l, ids.int().contiguous(), "softmax", False)
        dp = torch.zeros_like(p).scatter_add(1, ids, dw.double())
        check(dl, l, ids, None, p, dp)
