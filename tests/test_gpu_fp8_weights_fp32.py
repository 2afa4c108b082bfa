"""Codes of FP32 weights: the real quotient 448 w / amax rounded once, also where it
lies next to the border between two codes.  64-bit arithmetic decides that: 448 w
holds 27 bits, a border times amax 29, so they are equal or differ by at least
2^-29 of their value, and a 64-bit quotient stays on its side of the border."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8
from test_gpu_fp8 import FLOOR, round_e4m3
from test_gpu_tokens import normal

pytestmark = pytest.mark.gpu


def expected(w):
    E, N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    p = torch.zeros((E, nb * 128, kb * 128), dtype=torch.float64, device="cuda")
    p[:, :N, :K] = w.double()
    b = p.view(E, nb, 128, kb, 128)
    a = b.abs().amax((2, 4)).clamp(min=FLOOR)
    q = round_e4m3(b * 448 / a[:, :, None, :, None]).view(E, nb * 128, kb * 128)[:, :N, :K]
    return q, (a / 448).float()


def check(w):
    codes, scales = fp8.quantize_weights(w)
    q, s = expected(w)
    wrong = codes.double() != q
    assert not wrong.any(), (int(wrong.sum()), wrong.numel())
    assert torch.equal(scales, s)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -90, 2.0 ** -99, 2.0 ** 100])
def test_next_to_every_border(scale):
    """Each block: one amax, weights within two steps of FP32 of a border."""
    v = np.arange(127, dtype=np.uint8)
    values = torch.from_numpy(v).view(torch.float8_e4m3fn).double().numpy()
    border = (values[:-1] + values[1:]) / 2
    g = np.random.default_rng(5)
    n = 6
    a = (1 + g.integers(0, 2 ** 23, (n, n)) / 2 ** 23).astype(np.float32)
    a[0] = np.float32(1.75)                        # exact ties
    b = border[g.integers(0, len(border), (n * 128, n * 128))]
    at = a.repeat(128, 0).repeat(128, 1).astype(np.float64) * b / 448
    w = at.astype(np.float32)
    for _ in range(2):
        step = g.integers(-1, 2, w.shape)
        w = np.where(step == 0, w, np.nextafter(w, np.where(step < 0, 0, 4).astype(np.float32)))
    w *= g.choice([-1, 1], w.shape).astype(np.float32)
    w[::128, ::128] = a
    check(torch.from_numpy(w * np.float32(scale))[None].cuda())


def test_normal_weights_of_ragged_sizes():
    check(normal(1, (2, 1500, 2064), torch.float32) * 0.02)
    check(normal(2, (1, 4096, 4096), torch.float32))


def test_infinite_or_missing_weights_make_their_products_nan():
    w = normal(1, (1, 128, 256), torch.float32)
    w[0, 3, 5] = float("inf")
    w[0, 7, 200] = float("nan")
    codes, scales = fp8.quantize_weights(w)
    y = fp8.linear(normal(2, (8, 256), torch.bfloat16), codes[0], scales[0])
    assert torch.isnan(y[:, 3]).all() and torch.isnan(y[:, 7]).all()
