"""The gate's order with a bias where 32-bit sums err by more than their neighbours differ: a
large score with a bias near minus itself keeps the large score's rounding, although its sum is as
small as the others'.  The order is that of the real sums, here in 64 bits.
"""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import gating

pytestmark = pytest.mark.gpu


def ids64(l, bias, topk, score):
    l = l.double()
    s = torch.softmax(l, 1) if score == "softmax" else 1 / (1 + torch.exp(-l))
    return torch.sort(s + bias.double(), dim=1, descending=True, stable=True).indices[:, :topk].int()


def test_a_large_score_behind_the_first_gap():
    l = torch.tensor([[-6.9067526, -6.9067607, 3.2739234]], device="cuda")
    bias = torch.tensor([0.0, 0.0, -0.9625233], device="cuda")
    for topk in (1, 2, 3):
        ids, _ = gating.topk_gate(l, topk, bias, "sigmoid")
        assert torch.equal(ids, ids64(l, bias, topk, "sigmoid"))
    assert gating.topk_gate(l, 1, bias, "sigmoid")[0].tolist() == [[2]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [3, 30, 100, 128, 200, 400, 900])
def test_large_scores_with_biases_against_them(E, score):
    """Half of the experts have large scores whose biases bring them to 0.001 up to rounding,
    the others scores of 0.001 without a bias."""
    g = torch.Generator().manual_seed(E)
    large = torch.arange(E) % 2 == 0
    if score == "sigmoid":
        base = torch.where(large, 6 * torch.rand(E, generator=g) - 1, torch.tensor(-6.9067548))
        s = torch.sigmoid(base.double())
    else:
        # a softmax shares one: few large ones, whose scores hold the others' sum too
        large = torch.arange(E) < 3
        base = torch.where(large, torch.rand(E, generator=g), torch.tensor(-6.0))
        s = torch.softmax(base.double(), 0)
    low = float(s[~large][0]) if bool((~large).any()) else 0.001
    bias = torch.where(large, low - s, torch.zeros_like(s)).float().cuda()
    T = 300
    jitter = torch.where(large, torch.tensor(3e-7), torch.tensor(3e-5)) * torch.randn((T, E), generator=g)
    l = (base + jitter).float().cuda()
    for topk in sorted({1, min(E, 2), min(E, 7), min(E, 32)}):
        ids, w = gating.topk_gate(l, topk, bias, score, False)
        assert torch.equal(ids, ids64(l, bias, topk, score))
        ref = (torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double()))
        ref = ref.gather(1, ids.long())
        assert bool(((w.double() - ref).abs() <= ref * 2 * (16 + 32) * 2.0 ** -24).all())


@pytest.mark.parametrize("below", [33.0, 50.0, 70.0, 85.0])
def test_small_softmax_scores_whose_argument_is_rounded(below):
    """l - max rounds by up to |l - max| * 2^-24: more than two neighbours' scores differ."""
    g = torch.Generator().manual_seed(int(below))
    E, T = 64, 300
    l = -below + 2e-5 * torch.randn((T, E), generator=g)
    l[:, 5] = 0.3 + 0.1 * torch.rand(T, generator=g)
    s = torch.exp(torch.tensor(-below, dtype=torch.float64))
    bias = (s * 1e-5 * torch.randn(E, generator=g).double()).float()
    bias[5] = -2.0
    l, bias = l.cuda(), bias.cuda()
    for topk in (1, 6, 20):
        ids, _ = gating.topk_gate(l, topk, bias, "softmax", False)
        assert torch.equal(ids, ids64(l, bias, topk, "softmax"))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_biases_that_are_not_finite(score):
    """What a bias of infinity takes out or puts first is certain, whatever the scores."""
    inf = float("inf")
    g = torch.Generator().manual_seed(2)
    for E in (40, 300):
        l = torch.randn((100, E), generator=g).cuda()
        bias = torch.randn(E, generator=g).mul_(0.05).cuda()
        bias[::3] = -inf
        bias[7] = inf
        for topk in (1, 8, 32):
            ids, w = gating.topk_gate(l, topk, bias, score, False)
            assert torch.equal(ids, ids64(l, bias, topk, score))
        bias[1:] = -inf                     # fewer left than chosen: the lowest numbers follow
        ids, w = gating.topk_gate(l, 4, bias, score, False)
        assert torch.equal(ids, ids64(l, bias, 4, score))
