"""RMS norm and its gradient without an eps, which the calls allow: rows that hold something
have a root mean square, and no row that is not there may reach the weight's gradient.

Tolerances as in test_gpu_norm.py: U of each term for the sums of a row, the rounding of the
outputs, and one addition of FP32 for each row of the weight's gradient.
"""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import norm
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

pytestmark = pytest.mark.gpu

U = 40 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def half_step(t):
    return torch.finfo(t).eps / 2


def inside(t, off):
    """A copy of t (dense) that begins `off` elements after a multiple of 16 bytes."""
    flat = torch.empty(t.numel() + off + 64, dtype=t.dtype, device="cuda")
    view = flat[off:off + t.numel()].view(t.shape)
    view.copy_(t)
    return view


# Narrow rows share a block: T is no multiple of a block's rows in any of these.
@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("kind,off", [("bf16", 0), ("fp16", 0), ("fp32", 0), ("bf16", 3), ("fp32", 1)])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 64), (9, 64), (3, 512), (1021, 257), (333, 1000),
                                 (611, 1536), (2, 6144)])
def test_gradient_without_eps(T, D, kind, off, dh):
    g = torch.Generator().manual_seed(31 * T + D)
    h, dy, add = (inside((torch.randn((T, D), generator=g) + 0.01).to(TYPES[kind]).cuda(), off)
                  for _ in range(3))
    assert bool((h.abs().amax(1) > 0).all())
    add = add if dh else None
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    around = torch.full((T * D + off + 64,), 7.0, dtype=h.dtype, device="cuda")
    dx, dw = around[off:off + T * D].view(T, D), torch.empty(D, device="cuda")
    ws = torch.empty(F.nvfp4_rms_norm_grad_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
    F.nvfp4_rms_norm_grad(dy, h, add, w, 0.0, dx, dw, ws)
    h64, dy64 = h.double(), dy.double()
    r = 1 / h64.square().mean(1, keepdim=True).sqrt()
    g64 = dy64 * w.double()
    more = 0.0 if add is None else add.double()
    ref = r * (g64 - h64 * r.square() * (g64 * h64).mean(1, keepdim=True)) + more
    size = r * (g64.abs() + h64.abs() * r.square() * (g64 * h64).abs().mean(1, keepdim=True)) \
        + (0.0 if add is None else add.double().abs())
    t = h.dtype
    assert bool(((dx.double() - ref).abs() <= ref.abs() * half_step(t) + 2 * U * size + TINY[t]).all())
    terms = dy64 * h64 * r
    assert bool(((dw.double() - terms.sum(0)).abs()
                 <= ((T + 64) * 2.0 ** -24 + U) * terms.abs().sum(0)).all())
    assert bool((around[:off] == 7).all()) and bool((around[off + T * D:] == 7).all())


@pytest.mark.parametrize("T,D", [(1, 64), (9, 64), (700, 257), (3, 2048)])
def test_python_calls_without_eps(T, D):
    g = torch.Generator().manual_seed(T + D)
    x = torch.randn((T, D), generator=g).cuda().requires_grad_()
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda().requires_grad_()
    dy = torch.randn((T, D), generator=g).cuda()
    y = norm.rms_norm(x, w, eps=0.0)
    x64, w64 = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    ref = x64 / x64.square().mean(1, keepdim=True).sqrt() * w64
    assert bool(((y.double() - ref).abs() <= ref.abs() * (2.0 ** -24 * (1 + U) + U)).all())
    got = torch.autograd.grad(y, (x, w), dy)
    want = torch.autograd.grad(ref, (x64, w64), dy.double())
    assert bool(((got[0].double() - want[0]).abs()
                 <= 2 * U * (want[0].abs() + want[0].abs().amax(1, keepdim=True))).all())
    terms = (dy.double() * x64 / x64.square().mean(1, keepdim=True).sqrt()).abs().sum(0)
    assert bool(((got[1].double() - want[1]).abs() <= ((T + 64) * 2.0 ** -24 + U) * terms).all())
