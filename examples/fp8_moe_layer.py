"""An MoE layer with FP8 experts, served and differentiated.

    python examples/fp8_moe_layer.py [--tokens 256] [--experts 16] [--hidden 1024] [--inner 512]

Serving: route, gate_up products with the tokens gathered while they are
quantised, SiLU(gate) * up quantised into the down products, weighted sum back in
token order (moe.Fp8MLP).  Training with frozen experts: the gradients of the
routing weights and of the tokens -- through the combine, the down product over
transposed weights, the gate's elementwise derivative, the gate_up product over
transposed weights and the gather -- and a step of the router along them.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_grouped_gemm_nvfp4_gb300 import fp8, moe, tokens  # noqa: E402


class FrozenExperts(torch.autograd.Function):
    """The experts' rows y [R, hidden] of dispatched rows, differentiable in the
    rows: the weights are FP8 and frozen, their transposes prepared once."""

    @staticmethod
    def forward(ctx, rows, layer, transposed, offsets):
        gate_up = fp8.expert_linear(rows, *layer.gate_up, offsets)
        ctx.save_for_backward(gate_up, offsets)
        ctx.transposed = transposed
        return fp8.expert_linear(gate_up, *layer.down, offsets, silu_mul=True)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        gate_up, offsets = ctx.saved_tensors
        gate_up_t, down_t = ctx.transposed
        dh = fp8.expert_linear(dy, *down_t, offsets).float()
        gate, up = gate_up.float().chunk(2, dim=1)
        s = torch.sigmoid(gate)
        dgate = dh * up * s * (1 + gate * (1 - s))
        dgu = torch.cat([dgate, dh * gate * s], dim=1).to(dy.dtype)
        return fp8.expert_linear(dgu, *gate_up_t, offsets), None, None, None


def layer_forward(x, router, layer, transposed, topk):
    """Tokens through router and experts, differentiable in x and router."""
    probs, ids = torch.softmax(x.float() @ router, dim=1).topk(topk, dim=1)
    weights = probs / probs.sum(1, keepdim=True)
    offsets, pos = layer.route(ids.to(torch.int32))
    rows = tokens.dispatch(x, pos, offsets)
    y = FrozenExperts.apply(rows, layer, transposed, offsets)
    return tokens.combine(y, pos, weights, offsets)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    w1 = randn(a.experts, 2 * a.inner, a.hidden) * a.hidden ** -0.5
    w2 = randn(a.experts, a.hidden, a.inner) * a.inner ** -0.5
    layer = moe.Fp8MLP(fp8.quantize_weights(w1), fp8.quantize_weights(w2))
    transposed = (fp8.transpose_weights(*layer.gate_up), fp8.transpose_weights(*layer.down))
    x = randn(a.tokens, a.hidden).to(torch.bfloat16)
    router = randn(a.hidden, a.experts) * a.hidden ** -0.5
    target = randn(a.tokens, a.hidden)

    # serving
    probs, ids = torch.softmax(x.float() @ router, dim=1).topk(a.topk, dim=1)
    out = layer.step(x, ids.to(torch.int32), probs / probs.sum(1, keepdim=True))
    print(f"served {a.tokens} tokens: out {tuple(out.shape)}, rms {out.float().square().mean().sqrt():.4f}")

    # a few steps of the router along its gradient
    router.requires_grad_()
    losses = []
    for _ in range(8):
        loss = (layer_forward(x, router, layer, transposed, a.topk).float() - target).square().mean()
        g, = torch.autograd.grad(loss, router)
        losses.append(loss.item())
        with torch.no_grad():
            router -= 0.05 * g / g.square().mean().sqrt() * router.square().mean().sqrt()
    print("loss " + " ".join(f"{v:.5f}" for v in losses))
    return losses


if __name__ == "__main__":
    main()
