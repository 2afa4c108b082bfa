"""RMS norm with residual, its 8-bit form and its gradient against 64-bit arithmetic.

Tolerances.  The sum of squares adds at most 16 elements in a thread, then at most ten
times two values, so its relative error is below 30 * 2^-24; rstd, the quotient and the
products add less than 10 roundings: U = 40 * 2^-24 of each term.  The output adds
half a step of its type.
"""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8, norm
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

pytestmark = pytest.mark.gpu

U = 40 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
#: spacing of the smallest numbers, half of it (FP16 outputs may be subnormal)
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def half_step(t):
    return torch.finfo(t).eps / 2


def rows(gen, T, D, kind, sigma=1.0, pad=0):
    x = torch.randn((T, D + pad), generator=gen).mul_(sigma).to(TYPES[kind]).cuda()
    return x[:, :D]


def y64(h, w, eps):
    h, w = h.double(), w.double()
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * w


CASES = [(1, 1, "bf16", 0), (1, 7, "fp16", 0), (3, 64, "bf16", 0), (1, 6144, "bf16", 0),
         (5, 6144, "fp32", 0), (400, 1536, "bf16", 0), (333, 2047, "fp16", 0),
         (700, 257, "fp32", 3), (310, 4104, "bf16", 8), (2, 16384, "bf16", 0),
         (2, 16383, "fp16", 1), (330, 8192, "fp16", 0), (320, 9000, "bf16", 0),
         (2000, 33, "bf16", 0), (306, 100, "fp32", 0), (0, 128, "bf16", 0)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,D,kind,pad", CASES)
def test_norm(T, D, kind, pad, residual):
    g = torch.Generator().manual_seed(D)
    x = rows(g, T, D, kind, 1.0, pad)
    r = rows(g, T, D, kind, 3.0, pad) if residual else None
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    if D % 2:
        w = w.to(TYPES[kind])
    out = norm.rms_norm(x, w, r, eps=1e-5)
    y, h = out if residual else (out, x)
    if residual:
        assert torch.equal(h, (x.float() + r.float()).to(x.dtype))
    ref = y64(h, w, 1e-5)
    t = x.dtype
    assert y.dtype == t and y.shape == x.shape
    assert bool(((y.double() - ref).abs() <= ref.abs() * (half_step(t) * (1 + U) + U) + TINY[t]).all())
    assert F.nvfp4_device_status() == F.NVFP4_OK


def e4m3_values(codes):
    return codes.double() if codes.dtype == torch.float64 else codes.float().double()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,D,kind,pad", [(1, 16, "bf16", 0), (1, 6144, "bf16", 0),
                                          (9, 144, "fp16", 8), (400, 1040, "bf16", 0),
                                          (310, 4096, "fp16", 16), (3, 16384, "bf16", 0),
                                          (320, 9232, "bf16", 0), (0, 256, "bf16", 0)])
def test_norm_fp8(T, D, kind, pad, residual):
    g = torch.Generator().manual_seed(D + 1)
    x = rows(g, T, D, kind, 1.0, pad)
    r = rows(g, T, D, kind, 2.0, pad) if residual else None
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(TYPES[kind]).cuda()
    out = norm.rms_norm_fp8(x, w, r)
    codes, scales = out[:2]
    h = x
    if residual:
        h = out[2]
        assert torch.equal(h, (x.float() + r.float()).to(x.dtype))
    nb = -(-D // 128)
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == (T, D)
    assert scales.shape == (nb, T) and scales.dtype == torch.float32
    ref = torch.nn.functional.pad(y64(h, w, 1e-6), (0, nb * 128 - D)).view(T, nb, 128)
    amax = ref.abs().amax(2)
    assert bool(((scales.t().double() - amax / 448).abs() <= amax / 448 * (U + 2.0 ** -23)).all())
    q = ref * 448 / amax.clamp(min=2.0 ** -100)[:, :, None]
    got = torch.nn.functional.pad(e4m3_values(codes), (0, nb * 128 - D)).view(T, nb, 128)
    # half a step of E4M3 (2^-4 of a normal value, 2^-10 below 2^-6)
    assert bool(((got - q).abs() <= (q.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) + 2 * U * q.abs()).all())


def test_norm_fp8_rows_of_zeros_and_not_finite():
    x = torch.randn((4, 256), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    w = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    clean = norm.rms_norm_fp8(x[:1], w)
    codes, scales = norm.rms_norm_fp8(x, w)
    assert torch.equal(codes[:1].view(torch.uint8), clean[0].view(torch.uint8))
    assert bool((codes[1].float() == 0).all()) and bool(torch.isfinite(scales[:, 1]).all())
    assert bool(torch.isnan(codes[2].float()).all())
    # an infinite row has rstd 0: inf * 0 at its place, zeros elsewhere
    y = norm.rms_norm(x, w)
    assert bool(torch.isnan(y[3, 200])) and bool((y[3, :200] == 0).all())
    assert bool(torch.isnan(codes[3, 200].float()))
    wq, ws = fp8.quantize_weights(torch.randn((64, 256), device="cuda"))
    out = fp8.linear_codes(codes, scales, wq, ws)
    assert bool(torch.isfinite(out[:2]).all()) and bool(torch.isnan(out[2]).all())


@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("T,D,kind,pad", CASES)
def test_norm_grad(T, D, kind, pad, dh):
    g = torch.Generator().manual_seed(D + 2)
    h, dy = rows(g, T, D, kind, 2.0, pad), rows(g, T, D, kind, 1.0, pad)
    dh = rows(g, T, D, kind, 1.0, pad) if dh else None
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    if D % 2:
        w = w.to(TYPES[kind])
    dx, dw = norm.rms_norm_grad(dy, h, w, dh, eps=1e-5)
    h64, dy64, w64 = h.double(), dy.double(), w.double()
    r = 1 / torch.sqrt(h64.square().mean(1, keepdim=True) + 1e-5)
    gr = dy64 * w64
    back = h64 * r ** 3 * (gr * h64).mean(1, keepdim=True)
    add = dh.double() if dh is not None else torch.zeros_like(h64)
    ref = r * gr - back + add
    size = r * gr.abs() + h64.abs() * r ** 3 * (gr * h64).abs().mean(1, keepdim=True) + add.abs()
    t = h.dtype
    assert bool(((dx.double() - ref).abs() <= ref.abs() * half_step(t) + 2 * U * size + TINY[t]).all())
    terms = dy64 * h64 * r
    bound = (T + 64) * 2.0 ** -24 * terms.abs().sum(0) + U * terms.abs().sum(0)
    rw = terms.sum(0)
    assert dw.dtype == w.dtype
    assert bool(((dw.double() - rw).abs() <= rw.abs() * half_step(w.dtype) + bound + TINY[w.dtype]).all())
    again = norm.rms_norm_grad(dy, h, w, dh, eps=1e-5)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("residual", [False, True])
def test_norm_autograd_against_differences(residual):
    """Gradients in every input, by the formula and by differences of the 64-bit norm."""
    g = torch.Generator().manual_seed(5)
    shape = (2, 3, 40)
    x = torch.randn(shape, generator=g).cuda().requires_grad_()
    r = torch.randn(shape, generator=g).cuda().requires_grad_() if residual else None
    w = (1 + 0.2 * torch.randn(40, generator=g)).cuda().requires_grad_()
    cy, ch = (torch.randn(shape, generator=g).cuda() for _ in range(2))

    def loss64(x, w, r):
        h = x.double() if r is None else x.double() + r.double()
        total = (y64(h, w, 1e-6) * cy.double()).sum()
        return total if r is None else total + (h * ch.double()).sum()

    out = norm.rms_norm(x, w, r)
    loss = (out * cy).sum() if r is None else (out[0] * cy).sum() + (out[1] * ch).sum()
    leaves = [x, w] + ([r] if residual else [])
    grads = torch.autograd.grad(loss, leaves)
    refs = torch.autograd.grad(loss64(x, w, r), leaves)
    for got, ref in zip(grads, refs):
        assert got.dtype == torch.float32
        # at most 6 rows and 40 columns: sums of values of order one
        assert bool(((got - ref).abs() <= 100 * U * (1 + ref.abs())).all())
    for i, leaf in enumerate(leaves):
        d = torch.randn(leaf.shape, generator=g).cuda().double()
        with torch.no_grad():
            args = [x.double(), w.double(), None if r is None else r.double()]
            plus, minus = list(args), list(args)
            plus[i], minus[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
            slope = (loss64(*plus) - loss64(*minus)) / 2e-5
            assert abs(float((grads[i].double() * d).sum() - slope)) <= 1e-4 * (1 + abs(float(slope)))
    # the sum alone
    if residual:
        gx, gr = torch.autograd.grad((norm.rms_norm(x, w, r)[1] * ch).sum(), (x, r))
        assert torch.equal(gx, ch) and torch.equal(gr, ch)


def test_norm_strides_alignment_streams_capture():
    g = torch.Generator().manual_seed(9)
    x = torch.randn((64, 300), generator=g).bfloat16().cuda()
    w = torch.randn(256, generator=g).bfloat16().cuda()
    ref = norm.rms_norm(x[:, :256].contiguous(), w)
    assert torch.equal(norm.rms_norm(x[:, :256], w), ref)
    odd = torch.empty((64, 301), dtype=torch.bfloat16, device="cuda")[:, 1:257]
    odd.copy_(x[:, :256])
    tol = ref.abs().float() * 2.0 ** -7           # another order of the sum: one step
    assert bool(((norm.rms_norm(odd, w).float() - ref.float()).abs() <= tol).all())
    turned = x[:, :256].t().contiguous().t()
    assert torch.equal(norm.rms_norm(turned, w), ref)
    assert torch.equal(norm.rms_norm(x[:1].expand(5, 300)[:, :256], w), ref[:1].expand(5, 256))
    codes = norm.rms_norm_fp8(x[:, :256].contiguous(), w)
    for view in (x[:, :256], odd, turned):
        got = norm.rms_norm_fp8(view, w)
        assert torch.equal(got[0].view(torch.uint8), codes[0].view(torch.uint8))
        assert torch.equal(got[1], codes[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = norm.rms_norm(x[:, :256], w, stream=side)
    raw = norm.rms_norm_fp8(x[:, :256], w, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(other, ref) and torch.equal(raw[1], codes[1])
    dy = torch.randn((64, 256), generator=g).bfloat16().cuda()
    eager = norm.rms_norm_grad(dy, x[:, :256], w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = norm.rms_norm(x[:, :256], w)
        dx, dw = norm.rms_norm_grad(dy, x[:, :256], w)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and torch.equal(dx, eager[0]) and torch.equal(dw, eager[1])


def test_linear_of_norm_codes():
    """The codes feed the product: as quantising the norm's rows inside it, up to the
    norm's own rounding to BF16 (2^-9 of a value) seen through E4M3 (2^-4 of a step)."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn((70, 400), generator=g).bfloat16().cuda()
    w = torch.ones(400, device="cuda", dtype=torch.bfloat16)
    wq, ws = fp8.quantize_weights(torch.randn((272, 400), generator=g).cuda())
    codes, scales = norm.rms_norm_fp8(x, w)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        y = fp8.linear_codes(codes, scales, wq, ws, dtype)
        assert y.dtype == dtype
        sq = scales.t().repeat_interleave(128, 1)[:, :400].double()
        sw = ws.repeat_interleave(128, 0)[:272].repeat_interleave(128, 1)[:, :400].double()
        ref = (codes.float().double() * sq) @ (wq.float().double() * sw).t()
        size = (codes.float().double() * sq).abs() @ (wq.float().double() * sw).abs().t()
        assert bool(((y.double() - ref).abs()
                     <= half_step(dtype) * ref.abs() + 400 * 2.0 ** -24 * size).all())


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [16384, 16383, 16382, 16381])
def test_widest_rows(D, kind):
    """Up to the limit of the width, also where a row begins inside a chunk of 16 bytes: the
    norm with residual and the gradient with dh, whose shared memory is then the largest."""
    g = torch.Generator().manual_seed(D)
    x, r, dy, dh = (rows(g, 5, D, kind) for _ in range(4))
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(TYPES[kind]).cuda()
    y, h = norm.rms_norm(x, w, r)
    ref = y64(h, w, 1e-6)
    t = x.dtype
    assert bool(((y.double() - ref).abs() <= ref.abs() * (half_step(t) * (1 + U) + U)).all())
    dx, dw = norm.rms_norm_grad(dy, h, w, dh)
    h6 = h.double().requires_grad_()
    w6 = w.double().requires_grad_()
    want, want_w = torch.autograd.grad(y64_graph(h6, w6), (h6, w6), dy.double())
    # dx: the terms' sizes, each with U; the mean of products has D of them
    rstd = 1 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + 1e-6)
    g6 = dy.double() * w.double()
    size = rstd * (g6.abs() + h.double().abs() * rstd.square()
                   * (g6 * h.double()).abs().mean(-1, keepdim=True)) + dh.double().abs()
    want = want + dh.double()
    assert bool(((dx.double() - want).abs() <= half_step(t) * want.abs() + 2 * U * size).all())
    size_w = (dy.double() * h.double() * rstd).abs().sum(0)
    assert bool(((dw.double() - want_w).abs()
                 <= half_step(t) * want_w.abs() + 2 * U * size_w).all())


def y64_graph(h, w):
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w


def inside(t, off):
    """A copy of t (dense) that begins `off` elements after a multiple of 16 bytes."""
    flat = torch.empty(t.numel() + off + 64, dtype=t.dtype, device="cuda")
    view = flat[off:off + t.numel()].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("kind,off", [("fp32", 1), ("bf16", 3), ("fp16", 7)])
@pytest.mark.parametrize("T,D", [(1, 8), (5, 256), (400, 256), (700, 512), (320, 4096),
                                 (3, 16384)])
def test_rows_begun_inside_a_chunk(T, D, kind, off):
    """The library's own calls on matrices that all begin inside 16 bytes, of widths that fill
    their threads: one chunk more a row.  Elements before and after y keep their values."""
    g = torch.Generator().manual_seed(D + off)
    x, r, dy, dh = (inside(rows(g, T, D, kind), off) for _ in range(4))
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    t = x.dtype
    around = [torch.full((T * D + off + 64,), 7.0, dtype=t, device="cuda") for _ in range(3)]
    h, y, dx = (a[off:off + T * D].view(T, D) for a in around)
    F.nvfp4_rms_norm(x, r, w, 1e-5, h, y)
    dw = torch.empty(D, device="cuda")
    ws = torch.empty(F.nvfp4_rms_norm_grad_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
    F.nvfp4_rms_norm_grad(dy, h, dh, w, 1e-5, dx, dw, ws)
    torch.cuda.synchronize()
    for a in around:
        assert bool((a[:off] == 7).all()) and bool((a[off + T * D:] == 7).all())
    assert torch.equal(h, (x.float() + r.float()).to(t))
    ref = y64(h, w, 1e-5)
    assert bool(((y.double() - ref).abs() <= ref.abs() * (half_step(t) * (1 + U) + U) + TINY[t]).all())
    # the aligned call differs in the order of its sums only
    ex, ew = norm.rms_norm_grad(dy.clone(), h.clone(), w, dh.clone(), eps=1e-5)
    rstd = 1 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + 1e-5)
    g6 = dy.double() * w.double()
    size = rstd * (g6.abs() + h.double().abs() * rstd.square()
                   * (g6 * h.double()).abs().mean(-1, keepdim=True)) + dh.double().abs()
    # (each is half a step from a value of its own, and those are 4 U of the sizes apart)
    assert bool(((dx.double() - ex.double()).abs()
                 <= 2 * half_step(t) * ex.double().abs() * 1.01 + 4 * U * size + 2 * TINY[t]).all())
    size_w = (dy.double() * h.double() * rstd).abs().sum(0)
    assert bool(((dw.double() - ew.double()).abs() <= 4 * U * size_w).all())


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("T,D", [(5, 8185), (5, 8192), (5, 8200), (400, 8200), (5, 12281),
                                 (310, 12288), (5, 12288), (5, 12304), (310, 12304)])
def test_rows_at_the_limits_of_a_block(T, D, kind):
    """Around the widths at which a row's threads take more elements each; few rows and many."""
    g = torch.Generator().manual_seed(T + D)
    x, r, dy = (rows(g, T, D, kind) for _ in range(3))
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(TYPES[kind]).cuda()
    t = x.dtype
    y, h = norm.rms_norm(x, w, r)
    ref = y64(h, w, 1e-6)
    assert bool(((y.double() - ref).abs() <= ref.abs() * (half_step(t) * (1 + U) + U)).all())
    ref = y64(x, w, 1e-6)
    assert bool(((norm.rms_norm(x, w).double() - ref).abs()
                 <= ref.abs() * (half_step(t) * (1 + U) + U)).all())
    dx, dw = norm.rms_norm_grad(dy, x, w)
    x6, w6 = x.double().requires_grad_(), w.double().requires_grad_()
    want, want_w = torch.autograd.grad(y64_graph(x6, w6), (x6, w6), dy.double())
    rstd = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
    g6 = dy.double() * w.double()
    size = rstd * (g6.abs() + x.double().abs() * rstd.square()
                   * (g6 * x.double()).abs().mean(-1, keepdim=True))
    assert bool(((dx.double() - want).abs() <= half_step(t) * want.abs() + 2 * U * size).all())
    size_w = (dy.double() * x.double() * rstd).abs().sum(0)
    assert bool(((dw.double() - want_w).abs()
                 <= half_step(t) * want_w.abs() + 2 * U * size_w).all())
    if kind == "bf16" and D % 16 == 0:
        codes, scales, h2 = norm.rms_norm_fp8(x, w, r)
        assert torch.equal(h2, h)
        ref = y64(h, w, 1e-6)
        wide = scales.double().repeat_interleave(128, 0)[:D].t()
        # half a step of E4M3: 2^-4 of the value, at least half the smallest step, 2^-10
        assert bool(((codes.float().double() * wide - ref).abs()
                     <= ref.abs() * 2.0 ** -4 * (1 + U) + 2.0 ** -10 * wide + U * ref.abs()).all())


@pytest.mark.parametrize("wtype", ["same", "fp32", "offset"])
@pytest.mark.parametrize("T,D,kind", [(1, 1, "bf16"), (1, 7, "fp16"), (1, 64, "bf16"),
                                      (4, 64, "fp16"), (1, 6144, "bf16"), (1, 6143, "fp16"),
                                      (2, 6144, "bf16"), (1, 2048, "fp32"), (1, 12288, "bf16"),
                                      (1, 12287, "fp32"), (3, 512, "bf16"), (9, 512, "fp32")])
def test_gradient_of_one_block(T, D, kind, wtype):
    """Rows of one block, whose weight sums are the result, and a few more; the weight (and so its
    gradient) of either type, or beginning inside 16 bytes."""
    g = torch.Generator().manual_seed(11 * T + D)
    x, dy, dh = (rows(g, T, D, kind) for _ in range(3))
    w = (1 + 0.3 * torch.randn(D, generator=g)).cuda()
    if wtype != "fp32":
        w = w.to(TYPES[kind])
    if wtype == "offset":
        w = inside(w, 1)
    dx, dw = norm.rms_norm_grad(dy, x, w, dh, eps=1e-5)
    assert dw.dtype == w.dtype and dw.shape == (D,)
    x6, w6 = x.double(), w.double()
    rstd = 1 / torch.sqrt(x6.square().mean(-1, keepdim=True) + 1e-5)
    g6 = dy.double() * w6
    back = x6 * rstd.square() * (g6 * x6).mean(-1, keepdim=True)
    want = rstd * (g6 - back) + dh.double()
    size = rstd * (g6.abs() + x6.abs() * rstd.square() * (g6 * x6).abs().mean(-1, keepdim=True)) \
        + dh.double().abs()
    assert bool(((dx.double() - want).abs()
                 <= half_step(x.dtype) * want.abs() + 2 * U * size + TINY[x.dtype]).all())
    terms = dy.double() * x6 * rstd
    want = terms.sum(0)
    assert bool(((dw.double() - want).abs() <= half_step(w.dtype) * want.abs()
                 + 2 * U * terms.abs().sum(0) + TINY[w.dtype]).all())
    again = norm.rms_norm_grad(dy, x, w, dh, eps=1e-5)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    # into the middle of a larger matrix: what lies beside the weight's gradient stays
    around = torch.full((D + 32,), 7.0, dtype=w.dtype, device="cuda")
    off = 1 if wtype == "offset" else 16
    ws = torch.empty(F.nvfp4_rms_norm_grad_workspace_bytes(T, D) + 4, dtype=torch.uint8,
                     device="cuda")[4:]
    F.nvfp4_rms_norm_grad(dy, x, dh, w, 1e-5, torch.empty_like(x), around[off:off + D], ws)
    assert torch.equal(around[off:off + D], dw)
    assert bool((around[:off] == 7).all()) and bool((around[off + D:] == 7).all())
