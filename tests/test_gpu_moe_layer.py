"""The MoE layer for a few tokens against 64-bit arithmetic with the same quantisation,
and the operators around it together.

Tolerance, in the norm.  The output's rounding is at most half a step of its type.
The products' FP32 sums err by about 1e-5 of a typical value, so of the codes of h
some 2 * 1e-5 / 2^-4 = 3e-4 land on the other side of a border, each off by at most an
eighth: sqrt(3e-4) / 8 = 2.2e-3 of the norm.
"""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8, gating, moe, norm
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

pytestmark = pytest.mark.gpu

FLIPS = 2.2e-3


def tolerance(t):
    return torch.finfo(t).eps / 2 + FLIPS


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def weights_of(g, E, N, K):
    w = (torch.randn((E, N, K), generator=g) * K ** -0.5).cuda()
    return fp8.quantize_weights(w)


def dequantised(pair):
    codes, scales = pair
    E, N, K = codes.shape
    s = scales.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return codes.float().double() * s


def quantised(x):
    """64-bit rows as the values that E4M3 codes with 1 x 128 scales stand for."""
    out = x.double().clone()
    for a in range(0, x.shape[1], 128):
        b = out[:, a:a + 128]
        amax = b.abs().amax(1, keepdim=True).clamp(min=2.0 ** -100)
        q = b * 448 / amax
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, a:a + 128] = torch.round(q / step) * step * (amax / 448)
    return out


def experts64(x, ids, weights, gate_up, down):
    """Ids outside the experts contribute nothing."""
    w1, w2 = dequantised(gate_up), dequantised(down)
    inner = w2.shape[2]
    xq = quantised(x)
    out = torch.zeros((x.shape[0], w2.shape[1]), dtype=torch.float64, device=x.device)
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if 0 <= e < w1.shape[0]:
                gu = w1[e] @ xq[t]
                h = torch.nn.functional.silu(gu[:inner]) * gu[inner:]
                out[t] += float(weights[t, k]) * (w2[e] @ quantised(h[None])[0])
    return out


SIZES = [(1, 1, 1, 16, 16, 16), (1, 8, 128, 512, 256, 512), (2, 2, 4, 1040, 528, 1040),
         (8, 8, 64, 256, 128, 272), (8, 4, 8, 400, 144, 130), (7, 16, 16, 256, 64, 100),
         (3, 2, 8, 128, 16, 8), (5, 8, 8, 2048, 1024, 2048), (7, 3, 300, 272, 48, 40),
         (6, 2, 1024, 144, 32, 24), (1, 2, 8, 4096, 2048, 4096), (4, 2, 4, 6144, 512, 512),
         (8, 5, 6, 80, 2000, 333), (8, 32, 64, 272, 144, 260), (6, 1, 5, 1024, 656, 1296),
         (1, 1, 2, 16, 4096, 16), (1, 1, 2, 8192, 16, 4096)]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,topk,E,K,inner,N", SIZES)
def test_layer(T, topk, E, K, inner, N, kind):
    g = torch.Generator().manual_seed(K + T)
    gate_up, down = weights_of(g, E, 2 * inner, K), weights_of(g, E, N, inner)
    x = torch.randn((T, K), generator=g).to(kind).cuda()
    router = (torch.randn((E, K), generator=g) * K ** -0.5).cuda()
    sigmoid = T % 2 == 0
    if sigmoid:
        router = router.to(kind)
    bias = torch.randn(E, generator=g).mul_(0.05).cuda() if sigmoid else None
    layer = moe.Fp8MoE(router, gate_up, down, topk, bias, "sigmoid" if sigmoid else "softmax",
                       renormalize=T % 3 != 0, scale=1.5)
    assert F.nvfp4_fp8_moe_layer_workspace_bytes(T, topk, E, K, inner, N) > 0
    out, ids, weights = layer.step_routed(x)
    logits = x.double() @ router.double().t()
    s = torch.sigmoid(logits) if sigmoid else torch.softmax(logits, 1)
    key = logits if bias is None else s + bias.double()
    rid = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :topk]
    assert torch.equal(ids.long(), rid)
    rw = s.gather(1, rid)
    if T % 3 != 0:
        rw = rw / rw.sum(1, keepdim=True)
    # logits of order one with errors below K * 2^-24 in the worst order
    assert bool(((weights.double() - 1.5 * rw).abs() <= 1.5 * rw * (K + 128) * 2.0 ** -24).all())
    ref = experts64(x, rid, 1.5 * rw, gate_up, down)
    assert out.dtype == kind and out.shape == (T, N)
    assert rel(out, ref) <= tolerance(kind)
    assert torch.equal(layer.step(x), out)                  # bit for bit
    assert F.nvfp4_device_status() == F.NVFP4_OK


def small(seed=0, T=6, topk=3, E=8, K=272, inner=144, N=200):
    g = torch.Generator().manual_seed(seed)
    gate_up, down = weights_of(g, E, 2 * inner, K), weights_of(g, E, N, inner)
    x = torch.randn((T, K), generator=g).bfloat16().cuda()
    return g, moe.Fp8MLP(gate_up, down), x


def test_given_routes():
    g, mlp, x = small()
    weights = torch.rand((6, 3), generator=g).cuda()
    ids = torch.rand((6, 8), generator=g).topk(3, dim=1).indices.to(torch.int32).cuda()
    out = mlp.step_few(x, ids, weights)
    assert rel(out, experts64(x, ids, weights, mlp.gate_up, mlp.down)) <= tolerance(x.dtype)
    # step() quantises what gate_up rounded to BF16: codes move by one step at most where
    # that crosses a border (2^-9 / 2^-4 of them by an eighth at most), and rounds rows
    assert rel(mlp.step(x, ids, weights), out.double()) <= 4 * 2.0 ** -8 + (2.0 ** -5) ** 0.5 / 8
    # everyone at one expert, in one place or another
    same = torch.tensor([[5, 0, 1]], dtype=torch.int32).expand(6, 3).contiguous().cuda()
    assert rel(mlp.step_few(x, same, weights),
               experts64(x, same, weights, mlp.gate_up, mlp.down)) <= tolerance(x.dtype)
    # an expert twice and three times
    twice = ids.clone()
    twice[0] = torch.tensor([4, 2, 4])
    twice[3] = 7
    assert rel(mlp.step_few(x, twice, weights),
               experts64(x, twice, weights, mlp.gate_up, mlp.down)) <= tolerance(x.dtype)
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_routes_that_are_none():
    g, mlp, x = small(1)
    weights = torch.rand((6, 3), generator=g).cuda()
    ids = torch.rand((6, 8), generator=g).topk(3, dim=1).indices.to(torch.int32).cuda()
    ids[1] = -1
    ids[2, 1] = 8
    ids[4, 2] = 1 << 20
    out = mlp.step_few(x, ids, weights)
    assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK
    assert bool((out[1] == 0).all())
    keep = [0, 2, 3, 4, 5]
    ref = experts64(x, ids, weights, mlp.gate_up, mlp.down)
    assert rel(out[keep], ref[keep]) <= tolerance(x.dtype)
    ids.fill_(-1)
    assert bool((mlp.step_few(x, ids, weights) == 0).all())
    assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK


def test_rows_that_are_not_finite_stay_alone():
    g, mlp, x = small(2)
    weights = torch.rand((6, 3), generator=g).cuda()
    ids = torch.rand((6, 8), generator=g).topk(3, dim=1).indices.to(torch.int32).cuda()
    clean = mlp.step_few(x, ids, weights)
    bad = x.clone()
    bad[2, 7] = float("nan")
    bad[4, 9] = float("inf")
    out = mlp.step_few(bad, ids, weights)
    assert bool(torch.isnan(out[[2, 4]]).all())
    keep = [0, 1, 3, 5]
    assert torch.equal(out[keep], clean[keep])
    router = torch.randn((8, 272), generator=g).cuda()
    layer = moe.Fp8MoE(router, mlp.gate_up, mlp.down, 3)
    a, b = layer.step(x), layer.step(bad)
    assert torch.equal(a[keep], b[keep]) and bool(torch.isnan(b[[2, 4]]).all())
    zero = x.clone()
    zero[1] = 0
    out = mlp.step_few(zero, ids, weights)
    assert bool((out[1] == 0).all()) and torch.equal(out[0], clean[0])
    # large rows: scales far from one
    big = (x.double() * 2.0 ** 100).to(torch.bfloat16)
    tiny = (x.double() * 2.0 ** -90).to(torch.bfloat16)
    for v in (big, tiny):
        one = mlp.step_few(v[:1], ids[:1], weights[:1])
        ref = experts64(v[:1], ids[:1], weights[:1], mlp.gate_up, mlp.down)
        if float(ref.abs().max()) < 3e38 and float(ref.abs().max()) > 1e-37:
            assert rel(one, ref) <= tolerance(v.dtype)


def test_strides_streams_capture_and_overlap():
    g, mlp, x = small(3)
    router = torch.randn((8, 272), generator=g).bfloat16().cuda()
    layer = moe.Fp8MoE(router, mlp.gate_up, mlp.down, 3)
    ref = layer.step(x)
    wide = torch.zeros((6, 301), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:273] = x
    assert torch.equal(layer.step(wide[:, 1:273]), ref)
    wide = torch.zeros((6, 304), dtype=torch.bfloat16, device="cuda")
    wide[:, :272] = x
    assert torch.equal(layer.step(wide[:, :272]), ref)
    assert torch.equal(layer.step(x.t().contiguous().t()), ref)
    assert torch.equal(moe.Fp8MoE(router.t().contiguous().t(), mlp.gate_up, mlp.down, 3).step(x), ref)
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(4):                       # calls on two streams may overlap
        for s in sides:
            s.wait_stream(torch.cuda.current_stream())
            outs.append(layer.step(x, stream=s))
    outs.append(layer.step(x, stream=sides[0].cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for gr in graphs:
        with torch.cuda.graph(gr):
            held.append(layer.step(x))
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in held)
    x.neg_()                                 # new tokens under the captured step
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], layer.step(x))


def test_more_tokens_than_one_launch_takes():
    """Many tokens take the general path; its choice is the gate's on FP32 logits."""
    g, mlp, _ = small(4)
    x = torch.randn((40, 272), generator=g).bfloat16().cuda()
    for router in (torch.randn((8, 272), generator=g).cuda(),
                   torch.randn((8, 272), generator=g).bfloat16().cuda()):
        layer = moe.Fp8MoE(router, mlp.gate_up, mlp.down, 2, score="sigmoid")
        out, ids, weights = layer.step_routed(x)
        few = torch.cat([layer.step(x[i:i + 8]) for i in range(0, 40, 8)])
        assert torch.equal(ids, torch.cat([layer.step_routed(x[i:i + 8])[1] for i in range(0, 40, 8)]))
        # rounding of gate_up to BF16 before the quantisation of h, and of the rows
        assert rel(out, few.double()) <= 4 * 2.0 ** -8 + (2.0 ** -5) ** 0.5 / 8
    assert layer.step(x[:0]).shape == (0, 200)
    assert mlp.step_few(x[:0], ids[:0], weights[:0]).shape == (0, 200)
    with pytest.raises(ValueError):
        mlp.step_few(x, ids, weights)
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_block_of_a_decoder():
    """Norm, layer, norm with 8-bit output, projection: as a decoding step calls them."""
    T, D, E, inner = 4, 256, 8, 128
    g = torch.Generator().manual_seed(11)
    gate_up, down = weights_of(g, E, 2 * inner, D), weights_of(g, E, D, inner)
    router = (torch.randn((E, D), generator=g) * D ** -0.5).cuda()
    w1, w2 = (1 + 0.1 * torch.randn((2, D), generator=g)).bfloat16().cuda()
    wq, ws = fp8.quantize_weights((torch.randn((384, D), generator=g) * D ** -0.5).cuda())
    layer = moe.Fp8MoE(router, gate_up, down, 2)
    attended = torch.randn((T, D), generator=g).bfloat16().cuda()
    stream0 = torch.randn((T, D), generator=g).bfloat16().cuda()

    def block(a, h):
        y, h = norm.rms_norm(a, w1, h)
        moved = layer.step(y)
        codes, scales, h = norm.rms_norm_fp8(moved, w2, h)
        return fp8.linear_codes(codes, scales, wq, ws), h, y

    out, h, y = block(attended, stream0)
    h1 = (attended.float() + stream0.float()).bfloat16().double()
    y64 = h1 / torch.sqrt(h1.square().mean(1, keepdim=True) + 1e-6) * w1.double()
    assert rel(y, y64) <= 2.0 ** -8
    ids, weights = gating.topk_gate(y.float() @ router.t(), 2)
    moved = experts64(y, ids, weights, gate_up, down)
    h2 = h1 + moved
    assert rel(h, h2) <= 2 * 2.0 ** -8 + FLIPS
    n2 = h2 / torch.sqrt(h2.square().mean(1, keepdim=True) + 1e-6) * w2.double()
    sw = ws.repeat_interleave(128, 0)[:384].repeat_interleave(128, 1)[:, :D].double()
    ref = n2 @ (wq.float().double() * sw).t()
    assert rel(out, ref) <= 2.0 ** -4 / 3 ** 0.5 + 4 * 2.0 ** -8      # the codes' rounding
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block(attended, stream0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured[0], out) and torch.equal(captured[1], h)


@pytest.mark.parametrize("T,topk,E,K,inner,N", [(8, 6, 96, 512, 2048, 512), (8, 8, 64, 256, 1024, 200),
                                                (1, 4, 16, 1024, 256, 4096), (3, 4, 32, 384, 512, 4864)])
def test_cuts_of_the_products(T, topk, E, K, inner, N):
    """Long items of few output columns, cut into many runs, and as many runs for each item."""
    test_layer(T, topk, E, K, inner, N, torch.bfloat16)
