"""Gate weights and their gradient where scores leave FP32's range: sigmoids of logits below
-87, softmax scores far below the largest, chosen by a bias.  Renormalised weights are the
scores' ratio, which does not.

Reference: the logarithms of the scores in 64 bits (log s = -log(1 + exp(-l)), or l), and their
softmax over the chosen.  Tolerance: an argument l - max is rounded once, |l - max| * 2^-24 of the
value, and functions, sum and quotient err by less than 32 steps; a subnormal value by two of
the smallest steps.
"""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import gating

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LEAST = 2.0 ** -149


def log_scores(l, score):
    return torch.nn.functional.logsigmoid(l.double()) if score == "sigmoid" else l.double()


def ratios(l, ids, score):
    return torch.softmax(log_scores(l, score).gather(1, ids.long()), 1)


def close(got, ref, l, factor=1.0):
    """l: logits of the same shape as ref, whose distances from the row's largest count."""
    far = (l.double() - l.double().amax(1, keepdim=True)).abs().clamp(max=110)
    return bool(((got.double() - ref).abs()
                 <= ref.abs() * factor * (far + 32) * 2.0 ** -24 + factor * 2 * LEAST).all())


def rows_of_logits(kind, E, g):
    """Rows around and below the smallest sigmoids that FP32 has."""
    centres = [-3.0, -80.0, -86.0, -87.5, -89.0, -95.0, -103.0, -104.5, -110.0, -500.0, -30000.0]
    l = torch.stack([c + 2 * torch.randn(E, generator=g) for c in centres])
    spread = -60.0 - 60.0 * torch.rand((40, E), generator=g)
    return torch.cat([l, spread]).to(TYPES[kind]).cuda()


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("E,topk", [(2, 2), (16, 1), (40, 6), (128, 8), (300, 32), (600, 5)])
@pytest.mark.parametrize("biased", [False, True])
def test_renormalised_sigmoids(E, topk, kind, biased):
    g = torch.Generator().manual_seed(E)
    l = rows_of_logits(kind, E, g)
    # a bias that decides alone: what is chosen is then known without the scores
    bias = torch.randperm(E, generator=g).float().cuda() if biased else None
    ids, w = gating.topk_gate(l, topk, bias, "sigmoid", True, 2.5)
    key = l.double() if bias is None else bias.double().expand(l.shape)
    want = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
    assert torch.equal(ids.long(), want)
    assert close(w, 2.5 * ratios(l, ids, "sigmoid"), l.gather(1, want))


def test_two_logits_below_the_range():
    l = torch.tensor([[-90.0, -91.0], [-200.0, -200.0]], device="cuda")
    ids, w = gating.topk_gate(l, 2, None, "sigmoid", True)
    e = torch.tensor([[1.0, -1.0], [0.0, 0.0]], dtype=torch.float64, device="cuda")
    ref = 1 / (1 + torch.exp(-e))
    assert ids.tolist() == [[0, 1], [0, 1]]
    assert bool(((w.double() - ref).abs() <= ref * 33 * 2.0 ** -24).all())


@pytest.mark.parametrize("E,topk", [(16, 4), (128, 8), (300, 8)])
def test_renormalised_softmax_scores_that_a_bias_chose(E, topk):
    """The largest logit is far above all that the bias lets through."""
    g = torch.Generator().manual_seed(E)
    for below in (50.0, 87.0, 100.0, 120.0, 3000.0):
        l = torch.randn((20, E), generator=g).cuda() - below
        l[:, 0] = 0.0
        bias = torch.randperm(E, generator=g).float().cuda()
        bias[0] = -1.0
        ids, w = gating.topk_gate(l, topk, bias, "softmax", True)
        want = torch.sort(bias, descending=True).indices[:topk]
        assert torch.equal(ids.long(), want.expand(20, topk))
        # (scores in FP32's range are taken as they are: their own arguments' rounding)
        far = below + 5 if below < 90 else 10
        ref = ratios(l, ids, "softmax")
        assert bool(((w.double() - ref).abs() <= ref * 2 * (far + 32) * 2.0 ** -24).all())


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_sigmoids_themselves_are_subnormal(kind):
    l = (-70.0 - 40.0 * torch.rand((50, 60), generator=torch.Generator().manual_seed(3))).to(TYPES[kind]).cuda()
    for topk in (8, 32):
        ids, w = gating.topk_gate(l, topk, None, "sigmoid", False)
        s = torch.exp(log_scores(l, "sigmoid")).gather(1, ids.long())
        assert bool(((w.double() - s).abs() <= s * 32 * 2.0 ** -24 + 2 * LEAST).all())
    # (the largest eight are normal numbers, the others not all)
    assert bool(((w > 0) & (w < 2.0 ** -126)).any())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("E,topk", [(2, 2), (16, 1), (40, 6), (128, 8), (300, 32), (600, 5)])
def test_gradient_of_renormalised_scores(E, topk, kind, score):
    g = torch.Generator().manual_seed(E + 1)
    l = rows_of_logits(kind, E, g)
    ids = torch.sort(l.double(), dim=1, descending=True, stable=True).indices[:, :topk].int()
    dw = torch.randn((l.shape[0], topk), generator=g).cuda()
    dl = gating.topk_gate_grad(dw, l, ids, score, True, 1.5)
    chosen = l.gather(1, ids.long())
    w, g64 = ratios(l, ids, score), 1.5 * dw.double()
    slope = torch.sigmoid(-chosen.double()) if score == "sigmoid" else torch.ones_like(w)
    # w_j (1 - s_j) sum_i w_i (g_j - g_i)
    pair = g64[:, :, None] - g64[:, None, :]
    ref = w * slope * (pair * w[:, None, :]).sum(2)
    far = (chosen.double() - chosen.double().amax(1, keepdim=True)).abs().clamp(max=110)
    size = w * slope * ((g64.abs() + (w * g64.abs()).sum(1, keepdim=True)) * (far.amax(1, keepdim=True) + 64))
    got = dl.double().gather(1, ids.long())
    step = torch.finfo(l.dtype).eps / 2
    assert bool(((got - ref).abs() <= ref.abs() * step + 2 * size * 2.0 ** -24 + 2 * LEAST
                 + (2.0 ** -134 if kind == "bf16" else 0.0)).all())
    assert topk == 1 or bool((got != 0).any(1).all())
    rest = dl.clone().scatter_(1, ids.long(), 0.0)
    assert bool((rest == 0).all())


def test_rows_of_nothing_stay_zero():
    inf = float("inf")
    l = torch.full((2, 20), -inf, device="cuda")
    l[1, 3] = -200.0
    for bias in (None, torch.zeros(20, device="cuda")):
        ids, w = gating.topk_gate(l, 4, bias, "sigmoid", True)
        assert ids.tolist() == [[0, 1, 2, 3], [3, 0, 1, 2]]
        assert w.tolist() == [[0.0] * 4, [1.0, 0.0, 0.0, 0.0]]
        dl = gating.topk_gate_grad(torch.ones_like(w), l, ids, "sigmoid", True)
        assert bool((dl == 0).all())
