"""RMS norm over many rows: blocks that walk three rows and more, so that the places of the rows
on their way are used again, in rows begun anywhere within 16 bytes too; and grids of several
rounds.  Tolerances as in test_gpu_norm.py.
"""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import norm
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

pytestmark = pytest.mark.gpu

U = 40 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def inside(t, off):
    flat = torch.empty(t.numel() + off + 64, dtype=t.dtype, device="cuda")
    view = flat[off:off + t.numel()].view(t.shape)
    view.copy_(t)
    return view


# 152 SMs take up to eight blocks each, of up to eight rows at a time
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,D,kind,off", [(8003, 2047, "fp16", 0), (2101, 6143, "bf16", 0),
                                          (1003, 12287, "bf16", 0), (1009, 16383, "bf16", 0),
                                          (905, 8191, "fp32", 0), (40009, 129, "bf16", 0),
                                          (4003, 2048, "bf16", 5), (5003, 6144, "bf16", 0),
                                          (20011, 1024, "fp16", 0), (5001, 4096, "fp32", 0)])
def test_many_rows(T, D, kind, off, residual):
    g = torch.Generator(device="cuda").manual_seed(T + D)

    def rows(sigma):
        return inside(torch.randn((T, D), generator=g, device="cuda").mul_(sigma).to(TYPES[kind]), off)

    x, r = rows(1.0), rows(2.0) if residual else None
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    t = x.dtype
    around = [torch.full((T * D + off + 64,), 7.0, dtype=t, device="cuda") for _ in range(2)]
    h, y = (a[off:off + T * D].view(T, D) for a in around)
    F.nvfp4_rms_norm(x, r, w, 1e-5, h if residual else None, y)
    torch.cuda.synchronize()
    assert bool((around[1][:off] == 7).all()) and bool((around[1][off + T * D:] == 7).all())
    for a in range(0, T, 4096):
        part = slice(a, a + 4096)
        if residual:
            assert torch.equal(h[part], (x[part].float() + r[part].float()).to(t))
        v = (h if residual else x)[part].double()
        ref = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5) * w.double()
        assert bool(((y[part].double() - ref).abs()
                     <= ref.abs() * (torch.finfo(t).eps / 2 * (1 + U) + U) + TINY[t]).all())


@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("T,D,kind,off", [(2101, 6143, "bf16", 0), (6007, 1001, "fp16", 0),
                                          (5003, 2048, "bf16", 5), (905, 8191, "fp32", 0)])
def test_gradient_of_many_rows(T, D, kind, off, dh):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    h, dy, add = (inside(torch.randn((T, D), generator=g, device="cuda").to(TYPES[kind]), off)
                  for _ in range(3))
    add = add if dh else None
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    t = h.dtype
    around = torch.full((T * D + off + 64,), 7.0, dtype=t, device="cuda")
    dx, dw = around[off:off + T * D].view(T, D), torch.empty(D, device="cuda")
    ws = torch.empty(F.nvfp4_rms_norm_grad_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
    F.nvfp4_rms_norm_grad(dy, h, add, w, 1e-5, dx, dw, ws)
    torch.cuda.synchronize()
    assert bool((around[:off] == 7).all()) and bool((around[off + T * D:] == 7).all())
    want = torch.zeros(D, dtype=torch.float64, device="cuda")
    size_w = torch.zeros_like(want)
    for a in range(0, T, 2048):
        part = slice(a, a + 2048)
        v, d = h[part].double(), dy[part].double()
        r = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5)
        gr, more = d * w.double(), 0.0 if add is None else add[part].double()
        ref = r * (gr - v * r.square() * (gr * v).mean(1, keepdim=True)) + more
        size = r * (gr.abs() + v.abs() * r.square() * (gr * v).abs().mean(1, keepdim=True)) \
            + (0.0 if add is None else more.abs())
        assert bool(((dx[part].double() - ref).abs()
                     <= ref.abs() * torch.finfo(t).eps / 2 + 2 * U * size + TINY[t]).all())
        want += (d * v * r).sum(0)
        size_w += (d * v * r).abs().sum(0)
    assert bool(((dw.double() - want).abs() <= ((T + 64) * 2.0 ** -24 + U) * size_w).all())


@pytest.mark.parametrize("T,D,kind", [(5003, 6144, "bf16"), (1007, 12304, "fp16"), (20011, 1024, "bf16")])
def test_codes_of_many_rows(T, D, kind):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    x, r = (torch.randn((T, D), generator=g, device="cuda").to(TYPES[kind]) for _ in range(2))
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(TYPES[kind])
    codes, scales, h = norm.rms_norm_fp8(x, w, r)
    for a in range(0, T, 4096):
        part = slice(a, a + 4096)
        assert torch.equal(h[part], (x[part].float() + r[part].float()).to(x.dtype))
        v = h[part].double()
        ref = v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6) * w.double()
        wide = scales[:, part].double().repeat_interleave(128, 0)[:D].t()
        # half a step of E4M3: 2^-4 of the value, at least half the smallest step, 2^-10
        assert bool(((codes[part].float().double() * wide - ref).abs()
                     <= ref.abs() * 2.0 ** -4 * (1 + U) + 2.0 ** -10 * wide + U * ref.abs()).all())
