"""FP8 block quantisers and products against 64-bit arithmetic.

Codes and scales are compared exactly (the 16-bit inputs' codes are defined by
the real quotient).  Products are compared with the 64-bit sum over the same
codes and scales: the output rounding, eps / 2 of the value, plus FP32 sums --
the tensor cores' over a K block (128 products, each addition at worst a
truncation, 2^-23 of the partial sum's largest term: 40 covers four steps of 32
joined by four additions) and one fused addition per K block -- so (nkb + 40) *
2^-23 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8, tokens
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F
from test_gpu_tokens import TINY, normal, routes

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -100


def e4m3_values():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return v


def round_e4m3(v):
    """64-bit |v| <= 448 to the nearest E4M3 value, ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def oracle_rows(x):
    """(E4M3 values, FP32 scales [kb, M]) of rows x."""
    M, K = x.shape
    kb = -(-K // 128)
    b = torch.nn.functional.pad(x.double(), (0, kb * 128 - K)).view(M, kb, 128)
    a = b.abs().amax(2).clamp(min=FLOOR)
    q = round_e4m3(b * 448 / a[:, :, None]).view(M, kb * 128)[:, :K]
    # (in 64 bits: torch divides FP32 by a number as a product with its reciprocal)
    return q, (a / 448).float().t().contiguous()


def product(q, s, w, ws):
    """64-bit product of codes and scales, and of their magnitudes."""
    N, K = w.shape
    wd = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    xd = q.double() * s.t().double().repeat_interleave(128, 1)[:, :K]
    return xd @ wd.t(), xd.abs() @ wd.abs().t()


def check(y, ref, mag, K, name=""):
    nkb = -(-K // 128)
    eps = torch.finfo(y.dtype).eps / 2
    allow = 1.01 * (eps * ref.abs() + (nkb + 40) * 2.0 ** -23 * mag) + TINY[y.dtype]
    err = (y.double() - ref).abs()
    assert torch.isfinite(y).all(), name
    assert (err <= allow).all(), (name, float((err / allow).max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (17, 1552), (64, 6144), (257, 512)])
def test_quantised_rows_are_exact(M, K, dtype):
    x = normal(M + K, (M, K), dtype)
    x[M // 2] *= 2.0 ** -7
    x[0, :16] = 0
    codes, scales = fp8.quantize_rows(x)
    q, s = oracle_rows(x)
    assert torch.equal(codes.double(), q)
    assert torch.equal(scales, s)


def test_quantiser_borders_ties_zeros_and_extremes():
    """Every bf16 mantissa against block maxima of every mantissa (exact ties
    occur where the maximum is a multiple of 7), zero and tiny blocks, and the
    largest finite values."""
    mant = 1 + torch.arange(128, dtype=torch.float64) / 128
    rows = []
    for m in range(128):
        for e in (0, -3, -9):
            r = mant * 2.0 ** e
            r = torch.where(torch.arange(128) % 2 == 0, r, -r)
            r[0] = mant[m] * 2
            rows.append(r)
    x = torch.stack(rows)
    x = torch.cat([x, x * 2.0 ** 100, x * 2.0 ** -90, torch.zeros(1, 128),
                   torch.full((1, 128), 2.0 ** -120),
                   torch.full((1, 128), float(torch.finfo(torch.bfloat16).max))])
    x = x.to(torch.bfloat16).cuda()
    codes, scales = fp8.quantize_rows(x)
    q, s = oracle_rows(x)
    assert torch.equal(codes.double(), q)
    assert torch.equal(scales, s)
    assert torch.isfinite(scales).all() and (scales > 0).all()


def test_quantise_to_routes_strides_and_silu():
    T, topk, E, K = 37, 4, 8, 272
    pos, off = routes(1, T, topk, E, 0.2)
    wide = normal(2, (T, 600), torch.bfloat16)
    x = wide[:, 8:8 + K]
    codes, scales = fp8.quantize_rows(x, pos)
    q, s = fp8.quantize_rows(x.contiguous())
    for k in range(topk):
        ok = pos[:, k] >= 0
        at = pos[ok, k].long()
        assert torch.equal(codes[at].view(torch.uint8), q[ok].view(torch.uint8))
        assert torch.equal(scales[:, at], s[:, ok])
    odd = wide[:, 3:3 + K]                       # unaligned base: copied first
    assert torch.equal(fp8.quantize_rows(odd)[0].view(torch.uint8),
                       fp8.quantize_rows(odd.contiguous())[0].view(torch.uint8))
    # SiLU(gate) * up in FP32: equal codes except next to a rounding border
    gu = normal(3, (T, 2 * K), torch.bfloat16) * 2
    codes, scales = fp8.quantize_rows(gu, silu_mul=True)
    g, u = gu[:, :K].double(), gu[:, K:].double()
    h = g / (1 + torch.exp(-g)) * u
    kb = -(-K // 128)
    b = torch.nn.functional.pad(h, (0, kb * 128 - K)).view(T, kb, 128)
    a = b.abs().amax(2).clamp(min=FLOOR)
    assert ((scales.t().double() - a / 448).abs() <= 4e-6 * a / 448).all()
    v = (b * 448 / a[:, :, None]).view(T, kb * 128)[:, :K]
    low, high = round_e4m3(v * (1 - 4e-6)), round_e4m3((v * (1 + 4e-6)).clamp(-448, 448))
    got = codes.double()
    assert ((got == low) | (got == high)).all()


def test_quantised_weights_are_exact():
    for E, N, K in ((1, 128, 128), (2, 100, 48), (3, 257, 400)):
        w = normal(E + N, (E, N, K), torch.bfloat16) * 0.02
        codes, scales = fp8.quantize_weights(w)
        nb, kb = -(-N // 128), -(-K // 128)
        p = torch.zeros((E, nb * 128, kb * 128), dtype=torch.float64, device="cuda")
        p[:, :N, :K] = w.double()
        b = p.view(E, nb, 128, kb, 128)
        a = b.abs().amax((2, 4)).clamp(min=FLOOR)
        q = round_e4m3(b * 448 / a[:, :, None, :, None]).view(E, nb * 128, kb * 128)[:, :N, :K]
        assert torch.equal(codes.double(), q)
        assert torch.equal(scales, (a / 448).float())
        tc, ts = fp8.transpose_weights(codes, scales)
        assert torch.equal(tc.double(), q.transpose(1, 2))
        assert torch.equal(ts, scales.transpose(1, 2))


def weights(seed, E, N, K):
    codes, scales = fp8.quantize_weights(normal(seed, (E, N, K), torch.float32) * 0.02)
    return codes, scales


# one token to several tiles of every width; ragged N and K; few units over a
# long K (the sum over a cluster) and many
DENSE = [(1, 128, 128), (1, 4096, 6144), (2, 1, 16), (2, 640, 1040), (3, 130, 272), (4, 4096, 6144),
         (4, 257, 8192), (7, 100, 48), (16, 256, 1024), (17, 130, 272),
         (32, 512, 4096), (33, 384, 144), (65, 1000, 528), (64, 128, 8192), (81, 257, 400),
         (129, 640, 1552), (333, 2056, 1552), (1000, 384, 256), (300, 6000, 128), (4000, 645, 272)]


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_linear(M, N, K, dtype):
    w, ws = weights(N + K, 1, N, K)
    w, ws = w[0], ws[0]
    x = normal(M, (M, K), dtype)
    y = fp8.linear(x, w, ws)
    ref, mag = product(*oracle_rows(x), w, ws)
    check(y, ref, mag, K)
    assert F.nvfp4_device_status() == F.NVFP4_OK


@pytest.mark.parametrize("M,N,K", [(50, 300, 1040), (3000, 333, 272), (2500, 1001, 128),
                                   (20000, 64, 144)])
def test_linear_output_types_strides_and_repeat(M, N, K):
    w, ws = weights(1, 1, N, K)
    x = normal(0, (M, K), torch.bfloat16)
    codes, scales = fp8.quantize_rows(x)
    ref, mag = product(codes, scales, w[0], ws[0])
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        wide = torch.full((M, N + 5), float("nan"), dtype=dtype, device="cuda")
        for c in (wide[:, :N], wide[:, 5:]):
            wide.fill_(float("nan"))
            F.nvfp4_fp8_gemm(codes, scales, w[0], ws[0], c)
            check(c, ref, mag, K)
            assert int(torch.isnan(wide).sum()) == 5 * M        # nothing else written
        first = c.clone()
        F.nvfp4_fp8_gemm(codes, scales, w[0], ws[0], c)
        assert torch.equal(first, c)
    y3 = fp8.linear(x.view(5, M // 5, K), w[0], ws[0])
    assert torch.equal(y3.view(M, N), fp8.linear(x, w[0], ws[0]))
    assert fp8.linear(x[:0], w[0], ws[0]).shape == (0, N)


def test_rows_with_nan_or_infinity_stay_alone():
    M, N, K = 40, 256, 512
    w, ws = weights(1, 1, N, K)
    x = normal(0, (M, K), torch.bfloat16)
    want = fp8.linear(x, w[0], ws[0])
    x[3, 200] = float("inf")
    x[31, 5] = float("nan")
    x[20] = 0
    y = fp8.linear(x, w[0], ws[0])
    assert torch.isnan(y[3]).all() and torch.isnan(y[31]).all() and not y[20].any()
    keep = [i for i in range(M) if i not in (3, 20, 31)]
    assert torch.equal(y[keep], want[keep])


def check_experts(x, w, ws, pos, off, R, gather, y):
    E, N, K = w.shape
    live = int(off[-1])
    if gather:
        rows = torch.zeros((R, K), dtype=x.dtype, device="cuda")
        for k in range(pos.shape[1]):
            ok = pos[:, k] >= 0
            rows[pos[ok, k].long()] = x[ok]
    else:
        rows = x
    q, s = oracle_rows(rows)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            ref, mag = product(q[a:b], s[:, a:b], w[e], ws[e])
            check(y[a:b], ref, mag, K, f"expert {e}")
    assert not y[live:].any()


# (T, topk, E, N, K): one token; every tile width; ragged N and K; experts
# without a token; the sum over a cluster
GROUPED = [(1, 1, 4, 128, 128), (1, 8, 8, 512, 2048), (5, 2, 16, 100, 144), (40, 4, 8, 257, 272),
           (64, 8, 16, 384, 256), (200, 2, 4, 130, 528), (300, 4, 8, 256, 400),
           (256, 8, 128, 256, 512), (700, 3, 5, 640, 128), (900, 5, 8, 1329, 400),
           (1500, 2, 4, 130, 144)]


@pytest.mark.parametrize("T,topk,E,N,K", GROUPED)
@pytest.mark.parametrize("dropped", [0.0, 0.25])
def test_expert_linear(T, topk, E, N, K, dropped):
    w, ws = weights(N, E, N, K)
    pos, off = routes(T + N, T, topk, E, dropped)
    R = T * topk
    for dtype, gather in ((torch.bfloat16, True), (torch.float16, False)):
        x = normal(K, (T if gather else R, K), dtype)
        y = fp8.expert_linear(x, w, ws, off, pos if gather else None)
        check_experts(x, w, ws, pos, off, R, gather, y)
    assert F.nvfp4_device_status() == F.NVFP4_OK


@pytest.mark.parametrize("T,topk,E,N,K", [(3, 4, 8, 130, 272), (50, 4, 8, 257, 400)])
def test_expert_linear_of_gated_halves(T, topk, E, N, K):
    """SiLU(gate) * up inside the call: the same codes as the quantiser's."""
    w, ws = weights(N, E, N, K)
    pos, off = routes(T + N, T, topk, E, 0.25)
    R = T * topk
    gu = normal(K, (R, 2 * K), torch.bfloat16) * 2
    gu[int(off[-1]):] = float("nan")
    y = fp8.expert_linear(gu, w, ws, off, silu_mul=True)
    codes, scales = fp8.quantize_rows(gu, silu_mul=True)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            ref, mag = product(codes[a:b], scales[:, a:b], w[e], ws[e])
            check(y[a:b], ref, mag, K, f"expert {e}")
    assert not y[int(off[-1]):].any()
    x = normal(1, (T, 2 * K), torch.bfloat16)       # gathered from token order as well
    rows = torch.zeros((R, 2 * K), dtype=torch.bfloat16, device="cuda")
    for k in range(topk):
        ok = pos[:, k] >= 0
        rows[pos[ok, k].long()] = x[ok]
    got = fp8.expert_linear(x, w, ws, off, pos, silu_mul=True)
    assert torch.equal(got, fp8.expert_linear(rows, w, ws, off, silu_mul=True))
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_few_routes_report_bad_routing():
    E, N, K, R = 4, 128, 256, 8
    w, ws = weights(3, E, N, K)
    x = normal(1, (R, K), torch.bfloat16)
    good = torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32).cuda()
    want = fp8.expert_linear(x, w, ws, good)
    y = fp8.expert_linear(x, w, ws, torch.tensor([0, 2, 4, 9, 8], dtype=torch.int32).cuda())
    assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK
    assert torch.equal(y[:4], want[:4])
    pos = torch.arange(R, dtype=torch.int32).view(4, 2).cuda()
    pos[3, 1] = R + 5
    fp8.expert_linear(x[:4], w, ws, good, pos)
    assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK
    assert F.nvfp4_device_status() == F.NVFP4_OK


def test_skewed_experts():
    """One expert with most rows, several with none, the first and last empty."""
    E, N, K, R = 9, 384, 656, 1500
    counts = [0, 1, 1200, 0, 0, 130, 129, 40, 0]
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    assert int(off[-1]) == R
    w, ws = weights(3, E, N, K)
    x = normal(1, (R, K), torch.bfloat16)
    y = fp8.expert_linear(x, w, ws, off)
    check_experts(x, w, ws, None, off, R, False, y)


def test_bad_offsets_are_reported():
    E, N, K, R = 4, 128, 256, 40
    w, ws = weights(3, E, N, K)
    x = normal(1, (R, K), torch.bfloat16)
    good = torch.tensor([0, 10, 20, 30, 40], dtype=torch.int32).cuda()
    want = fp8.expert_linear(x, w, ws, good)
    for bad in ([0, 10, 20, 50, 40], [-3, 10, 20, 30, 40], [0, 10, 20, 30, 50]):
        off = torch.tensor(bad, dtype=torch.int32).cuda()
        y = fp8.expert_linear(x, w, ws, off)
        assert F.nvfp4_device_status() == F.NVFP4_ERR_DEVICE_CHECK
        for e in range(E):                    # the monotone experts are computed
            if 0 <= bad[e] <= bad[e + 1] <= R and bad[e] == 10 * e and bad[e + 1] == 10 * e + 10:
                assert torch.equal(y[10 * e:10 * e + 10], want[10 * e:10 * e + 10])


def test_gradient_of_the_tokens_through_transposed_weights():
    """<dy, W x> differentiated: dx = dy . W over the transposed codes."""
    T, topk, E, N, K = 24, 2, 4, 256, 384
    w, ws = weights(5, E, N, K)
    wt, wst = fp8.transpose_weights(w, ws)
    pos, off = routes(4, T, topk, E)
    dy = normal(1, (T * topk, N), torch.bfloat16)
    dx = tokens.dispatch_grad(fp8.expert_linear(dy, wt, wst, off), pos)
    want = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    q, s = oracle_rows(dy)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            r, m = product(q[a:b], s[:, a:b], wt[e], wst[e])
            for k in range(topk):
                at = (pos[:, k] >= a) & (pos[:, k] < b)
                want[at] += r[pos[at, k].long() - a]
                mag[at] += m[pos[at, k].long() - a]
    # two bf16 roundings (the rows', the sum's)
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs()
            + (2.0 ** -8 + (2 + 40) * 2.0 ** -23 + 2.0 ** -22) * mag).all()


def test_streams_and_capture():
    T, topk, E, N, K = 32, 4, 8, 256, 512
    w, ws = weights(5, E, N, K)
    pos, off = routes(4, T, topk, E)
    x = normal(1, (T, K), torch.bfloat16)
    want, dense = fp8.expert_linear(x, w, ws, off, pos), fp8.linear(x, w[0], ws[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        a = fp8.expert_linear(x, w, ws, off, pos, stream=stream)
        b = fp8.linear(x, w[0], ws[0], stream=stream)
        side.synchronize()
        assert torch.equal(a, want) and torch.equal(b, dense)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = fp8.expert_linear(x, w, ws, off, pos)
        b = fp8.linear(x, w[0], ws[0])
    x.copy_(normal(2, (T, K), torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, fp8.expert_linear(x, w, ws, off, pos))
    assert torch.equal(b, fp8.linear(x, w[0], ws[0]))


@pytest.mark.parametrize("M,N,K", [(5, 128, 2048), (64, 20000, 256), (500, 512, 1024)])
def test_expired_wait_is_reported(M, N, K):
    """A stage that never fills: the kernel gives up within its limit, records
    it and returns; the next call is right again."""
    w, ws = weights(5, 1, N, K)
    x = normal(1, (M, K), torch.bfloat16)
    want = fp8.linear(x, w[0], ws[0])
    F.nvfp4_set_timeout_ns(20_000_000)
    F.nvfp4_debug_set_flags(1)
    try:
        fp8.linear(x, w[0], ws[0])
        torch.cuda.synchronize()
        assert F.nvfp4_device_status() == F.NVFP4_ERR_TIMEOUT
    finally:
        F.nvfp4_debug_set_flags(0)
        F.nvfp4_set_timeout_ns(1_000_000_000)
    assert torch.equal(fp8.linear(x, w[0], ws[0]), want)
    assert F.nvfp4_device_status() == F.NVFP4_OK
