"""The FP8 MoE layer: the calls together, its capture, and the gradients of the
example against 64-bit arithmetic over the dequantised weights.

The layer quantises activations twice (three bits after the leading one: at most
2^-4 of a value, 2^-4 / sqrt(3) in the root mean square for the worst place
within a binade), forward and again backward, so outputs and gradients are
compared in the norm: 2 * 2^-4 / sqrt(3) = 7.2%.
"""
import os
import sys

import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8, moe, tokens
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import fp8_moe_layer as example  # noqa: E402

pytestmark = pytest.mark.gpu

NOISE = 2 * 2.0 ** -4 / 3 ** 0.5


def layer_of(seed, E, N, K, inner):
    g = torch.Generator().manual_seed(seed)
    w1 = (torch.randn((E, 2 * inner, K), generator=g) * K ** -0.5).cuda()
    w2 = (torch.randn((E, N, inner), generator=g) * inner ** -0.5).cuda()
    return moe.Fp8MLP(fp8.quantize_weights(w1), fp8.quantize_weights(w2))


def dequantised(pair):
    codes, scales = pair
    E, N, K = codes.shape
    s = scales.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return codes.double() * s


def reference(x, ids, weights, w1, w2):
    """64-bit MoE MLP, differentiable."""
    inner = w2.shape[2]
    out = torch.zeros((x.shape[0], w2.shape[1]), dtype=torch.float64, device=x.device)
    for k in range(ids.shape[1]):
        e = ids[:, k].long()
        gu = torch.einsum("tk,tnk->tn", x, w1[e])
        h = torch.nn.functional.silu(gu[:, :inner]) * gu[:, inner:]
        out = out + weights[:, k, None] * torch.einsum("ti,tni->tn", h, w2[e])
    return out


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("T,topk,E,N,K,inner", [(1, 2, 4, 256, 256, 128), (70, 4, 8, 272, 400, 144),
                                                (300, 2, 4, 512, 256, 256)])
def test_layer(T, topk, E, N, K, inner):
    layer = layer_of(T, E, N, K, inner)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16).cuda()
    ids = torch.rand((T, E), generator=g).topk(topk, dim=1).indices.to(torch.int32).cuda()
    weights = torch.rand((T, topk), generator=g).cuda()
    out = layer.step(x, ids, weights)
    ref = reference(x.double(), ids, weights.double(), dequantised(layer.gate_up),
                    dequantised(layer.down))
    assert rel(out, ref) <= NOISE
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = layer.step(x, ids, weights, stream=side)
    side.synchronize()
    assert torch.equal(other, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer.step(x, ids, weights)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, out)
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_gradients_through_frozen_experts():
    T, topk, E, N, K, inner = 60, 3, 6, 256, 256, 128
    layer = layer_of(3, E, N, K, inner)
    transposed = (fp8.transpose_weights(*layer.gate_up), fp8.transpose_weights(*layer.down))
    g = torch.Generator().manual_seed(2)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16).cuda().requires_grad_()
    ids = torch.rand((T, E), generator=g).topk(topk, dim=1).indices.to(torch.int32).cuda()
    weights = torch.rand((T, topk), generator=g).cuda().requires_grad_()
    c = torch.randn((T, N), generator=g).cuda()
    offsets, pos = layer.route(ids)
    y = example.FrozenExperts.apply(tokens.dispatch(x, pos, offsets), layer, transposed, offsets)
    out = tokens.combine(y, pos, weights, offsets)
    gx, gw = torch.autograd.grad((out.float() * c).sum(), (x, weights))
    x64 = x.detach().double().requires_grad_()
    w64 = weights.detach().double().requires_grad_()
    ref = reference(x64, ids, w64, dequantised(layer.gate_up), dequantised(layer.down))
    rx, rw = torch.autograd.grad((ref * c.double()).sum(), (x64, w64))
    assert rel(gx, rx) <= 2 * NOISE          # the forward's noise and the backward's
    assert rel(gw, rw) <= NOISE


def test_example_runs_and_learns():
    losses = example.main(["--tokens", "96", "--experts", "8", "--hidden", "256", "--inner", "128"])
    assert losses[-1] < losses[0]


def test_layer_refuses_shapes_that_do_not_fit():
    a = torch.zeros((2, 256, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        moe.Fp8MLP((a, None), (a, None))
