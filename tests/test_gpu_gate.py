"""Top-k gate and its gradient against 64-bit arithmetic.

Tolerances.  A softmax score is exp(l - max), whose argument is rounded once (|l - max|
* 2^-24 of the value) and whose function and sum err by less than 16 steps of FP32; a
sigmoid likewise.  U(l) = (|l| range + 32) * 2^-24 of each value.
"""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import gating
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def scores64(l, score):
    l = l.double()
    return torch.softmax(l, 1) if score == "softmax" else 1 / (1 + torch.exp(-l))


def gate64(l, topk, bias, score, renormalize, scale):
    s = scores64(l, score)
    key = l.double() if bias is None else s + bias.double()
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
    w = s.gather(1, ids)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w * scale


def unit(l):
    return (float((l.max() - l.min()).clamp(max=90)) + 32) * 2.0 ** -24 if l.numel() else 0.0


CASES = [(1, 1, 1, "fp32"), (1, 128, 8, "fp32"), (3, 8, 8, "bf16"), (1021, 60, 6, "bf16"),
         (517, 64, 1, "fp16"), (700, 256, 8, "fp32"), (65, 257, 5, "fp16"), (33, 1024, 32, "fp32"),
         (100, 33, 32, "bf16"), (0, 16, 2, "fp32"), (4097, 128, 8, "fp32")]


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score,renormalize,scale", [("softmax", True, 1.0), ("softmax", False, 1.5),
                                                     ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)])
@pytest.mark.parametrize("T,E,topk,kind", CASES)
def test_gate(T, E, topk, kind, score, renormalize, scale, biased):
    g = torch.Generator().manual_seed(E + T)
    l = torch.randn((T, E + 3), generator=g).mul_(2).to(TYPES[kind]).cuda()[:, :E]
    bias = torch.randn(E, generator=g).mul_(0.05).cuda() if biased else None
    ids, w = gating.topk_gate(l, topk, bias, score, renormalize, scale)
    rid, rw = gate64(l, topk, bias, score, renormalize, scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert torch.equal(ids, rid)
    assert bool(((w.double() - rw).abs() <= rw * 2 * unit(l)).all())
    again = gating.topk_gate(l, topk, bias, score, renormalize, scale)
    assert torch.equal(again[0], ids) and torch.equal(again[1], w)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_number(score):
    l = torch.zeros((3, 70), device="cuda")
    l[1, 40:] = -0.0
    l[2, ::2] = 1.0
    for bias in (None, torch.zeros(70, device="cuda")):
        ids, _ = gating.topk_gate(l, 6, bias, score)
        assert ids.tolist() == [list(range(6)), list(range(6)), [0, 2, 4, 6, 8, 10]]


def test_order_of_scores_that_32_bits_cannot_tell_apart():
    """Saturated sigmoids differ by less than half a step of FP32 around 1, and the
    larger bias can lie on the smaller logit."""
    l = torch.tensor([[20.0, 21.0, 19.0, 22.0, 3.0, -100.0, 2.0, 1.0]], device="cuda")
    bias = torch.zeros(8, device="cuda")
    ids, w = gating.topk_gate(l, 4, bias, "sigmoid", renormalize=False)
    assert ids.tolist() == [[3, 1, 0, 2]]
    bias[2] = 2.0 ** -27                    # more than sigmoid(22) - sigmoid(19)
    ids, w = gating.topk_gate(l, 4, bias, "sigmoid", renormalize=False)
    assert ids.tolist() == [[2, 3, 1, 0]]
    assert bool((w == 1.0).all())
    g = torch.Generator().manual_seed(1)
    l = (12 + torch.rand((300, 128), generator=g)).cuda()
    bias = (torch.randint(0, 3, (128,), generator=g) * 2.0 ** -24).cuda()
    ids, _ = gating.topk_gate(l, 8, bias, "sigmoid")
    assert torch.equal(ids, gate64(l, 8, bias, "sigmoid", True, 1.0)[0])


@pytest.mark.parametrize("spread,E", [(1e-6, 128), (1e-7, 20), (3e-7, 300), (1e-5, 64)])
def test_order_of_clusters_nearer_than_rounding(spread, E):
    """Scores in clusters a few 32-bit steps wide, around the last chosen place too."""
    g = torch.Generator().manual_seed(E)
    centre = torch.randint(0, 6, (200, E), generator=g).float() * 0.5 - 1.5
    l = (centre + spread * torch.randn((200, E), generator=g)).cuda()
    bias = (spread * torch.randn(E, generator=g)).cuda()
    for score in ("sigmoid", "softmax"):
        for topk in (1, 7, 20):
            ids, w = gating.topk_gate(l, topk, bias, score, False)
            rid, rw = gate64(l, topk, bias, score, False, 1.0)
            assert torch.equal(ids, rid)
            assert bool(((w.double() - rw).abs() <= rw * 2 * unit(l)).all())


def test_masked_rows_infinities_and_nan():
    inf, nan = float("inf"), float("nan")
    l = torch.randn((8, 40), generator=torch.Generator().manual_seed(2)).cuda()
    l[1] = -inf                              # nothing left
    l[2, 3:] = -inf                          # fewer than topk left
    l[3, 7] = inf
    l[4, 9] = nan
    l[5] = torch.finfo(torch.float32).min
    l[6, 1:] = torch.finfo(torch.float32).min
    for renormalize in (True, False):
        ids, w = gating.topk_gate(l, 4, None, "softmax", renormalize)
        rid, rw = gate64(l, 4, None, "softmax", renormalize, 1.0)
        for t in (0, 2, 5, 6, 7):
            assert torch.equal(ids[t], rid[t])
            assert bool(((w[t].double() - rw[t]).abs() <= rw[t] * 130 * 2.0 ** -24).all())
        assert ids[1].tolist() == [0, 1, 2, 3] and bool((w[1] == 0).all())
        assert ids[3, 0] == 7 and bool(torch.isnan(w[3, 0]))
        assert ids[4, 0] == 9 and bool(torch.isnan(w[4, 0]))
    ids, w = gating.topk_gate(l, 4, None, "sigmoid", True)
    assert ids[1].tolist() == [0, 1, 2, 3] and bool((w[1] == 0).all())
    assert ids[3, 0] == 7 and bool(torch.isfinite(w[3]).all())
    # experts masked by a bias
    bias = torch.zeros(40, device="cuda")
    bias[:36] = -inf
    ids, w = gating.topk_gate(l[:1], 4, bias, "sigmoid", True)
    assert sorted(ids[0].tolist()) == [36, 37, 38, 39]
    ids, w = gating.topk_gate(l[:1], 6, bias, "softmax", True)
    assert sorted(ids[0, :4].tolist()) == [36, 37, 38, 39] and ids[0, 4:].tolist() == [0, 1]


@pytest.mark.parametrize("score,renormalize,scale", [("softmax", True, 1.0), ("softmax", False, 1.5),
                                                     ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)])
@pytest.mark.parametrize("T,E,topk,kind", CASES)
def test_gate_grad(T, E, topk, kind, score, renormalize, scale):
    g = torch.Generator().manual_seed(E + 7 * T)
    l = torch.randn((T, E + 5), generator=g).mul_(2).to(TYPES[kind]).cuda()[:, :E]
    dw = torch.randn((T, topk), generator=g).cuda()
    ids = gate64(l, topk, None, score, renormalize, scale)[0]
    dl = gating.topk_gate_grad(dw, l, ids, score, renormalize, scale)
    l64 = l.double().requires_grad_()
    s = scores64(l64, score)
    w = s.gather(1, ids.long())
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    ref, = torch.autograd.grad((w * scale * dw.double()).sum(), l64)
    assert dl.dtype == l.dtype and dl.shape == (T, E)
    # each value is a difference of terms no larger than p * max |dw| * scale (/ S)
    with torch.no_grad():
        s = scores64(l, score)
        chosen = s.gather(1, ids.long())
        p = s / chosen.sum(1, keepdim=True) if renormalize else s
        size = p * scale * dw.double().abs().sum(1, keepdim=True)
        step = torch.finfo(l.dtype).eps / 2
        tiny = 2.0 ** -25 if l.dtype == torch.float16 else 0.0
        assert bool(((dl.double() - ref).abs() <= ref.abs() * step + 4 * unit(l) * size + tiny).all())
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_gate_grad_ends():
    """Rows with nothing left, saturated sigmoids, an expert twice, one that is none."""
    inf = float("inf")
    l = torch.randn((4, 12), generator=torch.Generator().manual_seed(4)).cuda()
    l[1] = -inf
    l[2] = 18.0
    dw = torch.ones((4, 3), device="cuda")
    ids = torch.tensor([[0, 1, 2]] * 4, dtype=torch.int32, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            dl = gating.topk_gate_grad(dw, l, ids, score, renormalize)
            assert bool((dl[1] == 0).all()) and bool(torch.isfinite(dl).all())
    dl = gating.topk_gate_grad(dw, l, ids, "sigmoid", False)
    s = l[2, 0].double()
    slope = float(torch.exp(-s) / (1 + torch.exp(-s)) ** 2)
    assert abs(float(dl[2, 0]) - slope) <= 60 * 2.0 ** -24 * slope
    twice = torch.tensor([[5, 5, 2]] * 4, dtype=torch.int32, device="cuda")
    for score in ("softmax", "sigmoid"):
        l64 = l[:1].double().requires_grad_()
        w = scores64(l64, score).gather(1, twice[:1].long())
        ref, = torch.autograd.grad(w.sum(), l64)
        got = gating.topk_gate_grad(dw[:1], l[:1], twice[:1], score, False)
        assert bool(((got.double() - ref).abs() <= 64 * 2.0 ** -24).all())
    bad = torch.tensor([[12, -1, 2]], dtype=torch.int32, device="cuda")
    got = gating.topk_gate_grad(dw[:1], l[:1], bad, "sigmoid", False)
    assert bool((got[0, [0, 1, 3, 4, 5, 6, 7, 8, 9, 10, 11]] == 0).all()) and bool(got[0, 2] != 0)
    assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK
    assert F.nvfp4_device_status() == F.NVFP4_OK


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False),
                                               ("sigmoid", True)])
def test_gate_autograd_against_differences(score, renormalize):
    g = torch.Generator().manual_seed(8)
    l = torch.randn((6, 20), generator=g).cuda().requires_grad_()
    c = torch.randn((6, 3), generator=g).cuda()
    bias = torch.randn(20, generator=g).mul_(0.05).cuda()
    ids, w = gating.topk_gate(l, 3, bias, score, renormalize, 2.0)
    assert not ids.requires_grad
    grad, = torch.autograd.grad((w * c).sum(), l)
    d = torch.randn((6, 20), generator=g).cuda().double()

    def loss(x):
        s = scores64(x, score).gather(1, ids.long())
        s = s / s.sum(1, keepdim=True) if renormalize else s
        return float((s * 2.0 * c.double()).sum())

    with torch.no_grad():
        slope = (loss(l.double() + 1e-5 * d) - loss(l.double() - 1e-5 * d)) / 2e-5
    assert abs(float((grad.double() * d).sum()) - slope) <= 1e-4 * (1 + abs(slope))


def test_gate_streams_and_capture():
    l = torch.randn((50, 96), generator=torch.Generator().manual_seed(6)).cuda()
    ref = gating.topk_gate(l, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = gating.topk_gate(l, 4, stream=s)
        side.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    turned = l.t().contiguous().t()
    assert torch.equal(gating.topk_gate(turned, 4)[1], ref[1])
    dw = torch.ones((50, 4), device="cuda")
    eager = gating.topk_gate_grad(dw, l, ref[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = gating.topk_gate(l, 4)
        dl = gating.topk_gate_grad(dw, l, ids)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids, ref[0]) and torch.equal(w, ref[1]) and torch.equal(dl, eager)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,topk,kind", [(40, 512, 8, "fp32"), (9, 511, 32, "bf16"),
                                           (40, 513, 8, "fp16"), (3, 384, 6, "fp32")])
def test_gate_of_many_experts(T, E, topk, kind, score, renormalize, biased):
    test_gate(T, E, topk, kind, score, renormalize, 1.0, biased)
    test_gate_grad(T, E, topk, kind, score, renormalize, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_gradient_of_one_renormalised_weight_is_zero(kind, score):
    """The weight is 1 whatever the logits: its gradient is 0, without any rounding's residue."""
    g = torch.Generator().manual_seed(21)
    l = torch.randn((300, 40), generator=g).mul_(3).to(TYPES[kind]).cuda()
    dw = torch.randn((300, 1), generator=g).cuda()
    ids, w = gating.topk_gate(l, 1, score=score, renormalize=True)
    assert bool((w == 1).all())
    assert bool((gating.topk_gate_grad(dw, l, ids, score, True) == 0).all())
