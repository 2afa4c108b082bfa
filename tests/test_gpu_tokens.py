"""Token rows into expert order and back, and the gradients of both, against
64-bit sums.

Tolerances: an output rounded to type t is off by at most eps(t) / 2 of its
value; an FP32 sum of n products by at most (n + 1) * 2^-24 of the sum of their
magnitudes.  The dot products of the routing weights' gradient are summed by at
least 32 threads each, so n = D / 32 + 16 there.
"""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F
from moe_grouped_gemm_nvfp4_gb300 import tokens

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def routes(seed, T, topk, E, dropped=0.0):
    """(route_pos, expert_offsets) on the GPU, -1 for dropped routes."""
    g = np.random.default_rng(seed)
    ids = np.argsort(g.random((T, E)), axis=1)[:, :topk] if topk <= E else \
        g.integers(0, E, (T, topk))
    ids = np.where(g.random((T, topk)) < dropped, E, ids).reshape(-1)
    order = np.argsort(ids, kind="stable")
    pos = np.empty(T * topk, np.int32)
    pos[order] = np.arange(T * topk)
    pos[ids == E] = -1
    off = np.zeros(E + 1, np.int32)
    off[1:] = np.cumsum(np.bincount(ids, minlength=E + 1)[:E])
    return torch.from_numpy(pos.reshape(T, topk)).cuda(), torch.from_numpy(off).cuda()


def normal(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float32).to(dtype).cuda()


def within(got, ref, slack, dtype):
    allow = 1.01 * (torch.finfo(dtype).eps / 2 * ref.abs() + slack) + TINY[dtype]
    bad = (got.double() - ref).abs() > allow
    assert not bad.any(), (int(bad.sum()), float(((got.double() - ref).abs() / allow).max()))


def ref_combine(y, pos, w):
    """(sum, sum of magnitudes) in 64 bits."""
    T, topk = pos.shape
    out = torch.zeros((T, y.shape[1]), dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(out)
    for k in range(topk):
        ok = pos[:, k] >= 0
        term = w[ok, k, None].double() * y[pos[ok, k].long()].double()
        out[ok] += term
        mag[ok] += term.abs()
    return out, mag


# one token; narrow and odd widths (element and 16-byte accesses); more routes
# than are in flight at once; widths over one block's columns
SHAPES = [(1, 1, 1, 1), (1, 8, 8, 6144), (3, 2, 4, 7), (5, 9, 16, 24), (64, 8, 16, 130),
          (17, 4, 8, 512), (33, 17, 20, 2056), (2, 3, 8, 10000), (300, 8, 128, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,topk,E,D", SHAPES)
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_dispatch_and_back(T, topk, E, D, dtype, dropped):
    pos, off = routes(T * 31 + D, T, topk, E, dropped)
    x = normal(D, (T, D), dtype)
    out = tokens.dispatch(x, pos, off)
    want = torch.zeros((T * topk, D), dtype=dtype, device="cuda")
    for k in range(topk):
        ok = pos[:, k] >= 0
        want[pos[ok, k].long()] = x[ok]
    assert torch.equal(out, want)
    dout = normal(D + 1, (T * topk, D), dtype)
    live = int(off[-1])
    dout[live:] = float("nan")                 # never read
    dx = tokens.dispatch_grad(dout, pos)
    ones = torch.ones(pos.shape, dtype=torch.float32, device="cuda")
    ref, mag = ref_combine(dout, pos, ones)
    within(dx, ref, (topk + 1) * 2.0 ** -24 * mag, dtype)
    assert F.nvfp4_device_status() == F.NVFP4_OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,topk,E,D", SHAPES)
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_combine_and_its_gradient(T, topk, E, D, dtype, dropped):
    pos, off = routes(T * 17 + D, T, topk, E, dropped)
    y = normal(D, (T * topk, D), dtype)
    y[int(off[-1]):] = float("nan")            # never read
    w = torch.rand((T, topk), generator=torch.Generator().manual_seed(D)).cuda()
    w = torch.where(pos >= 0, w, torch.full_like(w, float("nan")))   # nor a dropped weight
    out = tokens.combine(y, pos, w)
    ref, mag = ref_combine(y, pos, w)
    within(out, ref, (topk + 1) * 2.0 ** -24 * mag, dtype)

    dout = normal(D + 2, (T, D), dtype)
    dy, dw = tokens.combine_grad(dout, y, pos, w, off)
    assert torch.equal(dy[int(off[-1]):], torch.zeros_like(dy[int(off[-1]):]))
    n = D / 32 + 16
    for k in range(topk):
        ok = pos[:, k] >= 0
        rows = pos[ok, k].long()
        d64 = dout[ok].double()
        want = w[ok, k, None].double() * d64
        within(dy[rows], want, 2.0 ** -24 * want.abs(), dtype)
        terms = d64 * y[rows].double()
        err = (dw[ok, k].double() - terms.sum(1)).abs()
        assert (err <= 1.01 * (n + 1) * 2.0 ** -24 * terms.abs().sum(1) + 1e-37).all()
        assert (dw[~ok, k] == 0).all()
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_results_repeat():
    pos, off = routes(5, 200, 8, 64, 0.1)
    y, dout = normal(1, (1600, 1024), torch.bfloat16), normal(2, (200, 1024), torch.bfloat16)
    w = torch.rand((200, 8)).cuda()
    first = (tokens.combine(y, pos, w), *tokens.combine_grad(dout, y, pos, w, off))
    for _ in range(3):
        again = (tokens.combine(y, pos, w), *tokens.combine_grad(dout, y, pos, w, off))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_no_live_route_and_no_token():
    pos = torch.full((5, 3), -1, dtype=torch.int32, device="cuda")
    off = torch.zeros(9, dtype=torch.int32, device="cuda")
    x = normal(0, (5, 64), torch.bfloat16)
    assert torch.equal(tokens.dispatch(x, pos, off), torch.zeros((15, 64)).bfloat16().cuda())
    y = torch.full((15, 64), float("inf")).bfloat16().cuda()
    w = torch.ones((5, 3)).cuda()
    assert torch.equal(tokens.combine(y, pos, w), torch.zeros((5, 64)).bfloat16().cuda())
    dy, dw = tokens.combine_grad(x, y, pos, w, off)
    assert not dy.any() and not dw.any()
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    assert tokens.dispatch(x[:0], none, off).shape == (0, 64)
    assert tokens.combine(y[:0], none, w[:0]).shape == (0, 64)
    dy, dw = tokens.combine_grad(x[:0], y[:0], none, w[:0], off)
    assert dy.shape == (0, 64) and dw.shape == (0, 3)


def test_infinities_pass_through():
    pos, off = routes(3, 4, 2, 4)
    y = normal(0, (8, 32), torch.float16)
    y[pos[1, 0].long(), 5] = float("inf")
    y[pos[2, 1].long(), 6] = float("nan")
    w = torch.full((4, 2), 0.5).cuda()
    out = tokens.combine(y, pos, w)
    assert torch.isinf(out[1, 5]) and torch.isnan(out[2, 6])
    assert int((~torch.isfinite(out)).sum()) == 2


@pytest.mark.parametrize("dtype", TYPES)
def test_row_strides_and_unaligned_bases(dtype):
    T, topk, E = 19, 4, 8
    pos, off = routes(7, T, topk, E)
    wide = normal(1, (T, 200), dtype)
    for x in (wide[:, 8:136], wide[:, 3:131], wide[:, 1:1 + 77]):
        want = tokens.dispatch(x.contiguous(), pos, off)
        assert torch.equal(tokens.dispatch(x, pos, off), want)
    yw = normal(2, (T * topk, 200), dtype)
    w = torch.rand((T, topk)).cuda()
    for sl in (slice(8, 136), slice(5, 133)):
        y, d = yw[:, sl], wide[:, sl]
        assert torch.equal(tokens.combine(y, pos, w), tokens.combine(y.contiguous(), pos, w))
        a = tokens.combine_grad(d, y, pos, w, off)
        b = tokens.combine_grad(d.contiguous(), y.contiguous(), pos, w, off)
        assert torch.equal(a[0], b[0])
        # the access width changes which thread sums which columns
        mag = 1.01 * (128 / 32 + 17) * 2.0 ** -23 * 128 * 16
        assert (a[1] - b[1]).abs().max() < mag
    # transposed rows and a broadcast gradient are copied first
    xt = normal(3, (64, T), dtype).t()
    assert torch.equal(tokens.dispatch(xt, pos, off), tokens.dispatch(xt.contiguous(), pos, off))
    one = torch.ones((), dtype=dtype, device="cuda").expand(T * topk, 64)
    assert torch.equal(tokens.dispatch_grad(one, pos),
                       torch.full((T, 64), topk, dtype=dtype, device="cuda"))


def test_positions_past_the_buffer_are_reported():
    pos, off = routes(3, 8, 2, 4)
    x = normal(0, (8, 64), torch.bfloat16)
    bad = pos.clone()
    bad[4, 1] = 16
    out = tokens.dispatch(x, bad)
    torch.cuda.synchronize()
    assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK
    ok = [i for i in range(16) if i != int(pos[4, 1])]
    assert torch.equal(out[ok], tokens.dispatch(x, pos, off)[ok])
    y = normal(1, (16, 64), torch.bfloat16)
    tokens.combine(y, bad, torch.ones((8, 2)).cuda())
    assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_offsets_past_32_bits():
    """Rows whose first element lies past 2^31 elements."""
    R, D, T = 70000, 32768, 3
    assert R * D > 2 ** 31
    pos = torch.tensor([[R - 1, 0], [5, R - 2], [R - 3, 7]], dtype=torch.int32, device="cuda")
    x = normal(0, (T, D), torch.bfloat16)
    out = tokens.dispatch(x, pos, R=R)
    for t in range(T):
        for k in range(2):
            assert torch.equal(out[int(pos[t, k])], x[t])
    w = torch.rand((T, 2)).cuda()
    got = tokens.combine(out, pos, w)
    ref, mag = ref_combine(out, pos, w)
    within(got, ref, 3 * 2.0 ** -24 * mag, torch.bfloat16)
    _, dw = tokens.combine_grad(x, out, pos, w)
    dot = (x.double() ** 2).sum(1, keepdim=True)
    assert ((dw.double() - dot).abs() <= 1.01 * (D / 32 + 17) * 2.0 ** -24 * dot).all()


def test_autograd_matches_the_formulas_and_differences():
    """Loss = <c, combine(f(dispatch(x)), w)> with f(r) = r * s per row, FP32."""
    T, topk, E, D = 6, 3, 5, 40
    pos, off = routes(11, T, topk, E, 0.2)
    x = normal(0, (T, D), torch.float32).requires_grad_()
    w = torch.rand((T, topk)).cuda().requires_grad_()
    s = normal(1, (T * topk, 1), torch.float32)
    c = normal(2, (T, D), torch.float32)

    def loss(x, w):
        return (tokens.combine(tokens.dispatch(x, pos, off) * s, pos, w, off) * c).sum()

    gx, gw = torch.autograd.grad(loss(x, w), (x, w))
    live = (pos >= 0)
    sp = s[pos.clamp(min=0).long(), 0].double() * live
    cx = (c.double() * x.detach().double()).sum(1, keepdim=True)
    want_w = sp * cx
    want_x = (w.detach().double() * sp).sum(1, keepdim=True) * c.double()
    assert torch.allclose(gw.double(), want_w, rtol=1e-5, atol=1e-5)
    assert torch.allclose(gx.double(), want_x, rtol=1e-5, atol=1e-5)
    # differences: the loss is linear in x and in w
    with torch.no_grad():
        for t, k in ((0, 0), (2, 1), (5, 2)):
            d = torch.zeros_like(w)
            d[t, k] = 0.5
            diff = (loss(x, w + d) - loss(x, w - d)).item()
            assert abs(diff - gw[t, k].item()) <= 1e-3 * (1 + abs(diff))
        d = torch.zeros_like(x)
        d[3, 7] = 0.5
        diff = (loss(x + d, w) - loss(x - d, w)).item()
        assert abs(diff - gx[3, 7].item()) <= 1e-3 * (1 + abs(diff))
    # a broadcast weight collects the gradient of every use
    one = torch.ones((), device="cuda", requires_grad=True)
    g, = torch.autograd.grad(loss(x.detach(), one.expand(T, topk)), one)
    assert abs(g.item() - want_w.sum().item()) <= 1e-4 * want_w.abs().sum().item()
    # y alone, without weights
    y = normal(4, (T * topk, D), torch.float32).requires_grad_()
    gy, = torch.autograd.grad((tokens.combine(y, pos, None, off) * c).sum(), y)
    assert torch.equal(gy, tokens.dispatch(c, pos, off))


def test_streams_and_capture():
    pos, off = routes(2, 64, 8, 16)
    x = normal(0, (64, 256), torch.bfloat16)
    w = torch.rand((64, 8)).cuda()
    want = tokens.combine(tokens.dispatch(x, pos, off), pos, w)
    grads = tokens.combine_grad(x, tokens.dispatch(x, pos, off), pos, w, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        y = tokens.dispatch(x, pos, off, stream=stream)
        got = tokens.combine(y, pos, w, stream=stream)
        g = tokens.combine_grad(x, y, pos, w, off, stream=stream)
        side.synchronize()
        assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(g, grads))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tokens.dispatch(x, pos, off)
        got = tokens.combine(y, pos, w)
        g = tokens.combine_grad(x, y, pos, w, off)
    x.copy_(normal(9, (64, 256), torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    y = tokens.dispatch(x, pos, off)
    assert torch.equal(got, tokens.combine(y, pos, w))
    assert all(torch.equal(a, b) for a, b in zip(g, tokens.combine_grad(x, y, pos, w, off)))
