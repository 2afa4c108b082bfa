"""An FP32 router's logits are FP32 whatever precision the process allows torch's own products,
for a few tokens and for many.

Tolerance: logits of order one whose FP32 sums err by less than K * 2^-24 in the worst order; the
weights by that, the exponentials' and the sums' 128 steps.
"""
import pytest
import torch

from test_gpu_moe_layer import weights_of

from moe_grouped_gemm_nvfp4_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.fixture
def tf32():
    before = torch.get_float32_matmul_precision()
    torch.set_float32_matmul_precision("high")
    yield
    torch.set_float32_matmul_precision(before)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [5, 9, 300])
def test_precision_of_the_choice(T, kind, tf32):
    E, K, inner, topk = 64, 1024, 16, 4
    g = torch.Generator().manual_seed(T)
    gate_up, down = weights_of(g, E, 2 * inner, K), weights_of(g, E, 16, inner)
    x = torch.randn((T, K), generator=g).to(kind).cuda()
    router = (torch.randn((E, K), generator=g) * K ** -0.5).cuda()
    layer = moe.Fp8MoE(router, gate_up, down, topk, score="sigmoid", renormalize=False)
    out, ids, weights = layer.step_routed(x)
    s = torch.sigmoid(x.double() @ router.double().t())
    ref = s.gather(1, ids.long())
    unit = (K + 128) * 2.0 ** -24
    assert bool(((weights.double() - ref).abs() <= ref * unit).all())
    # what is left out is no larger than what was chosen, up to the same error
    rest = s.scatter(1, ids.long(), 0.0).amax(1)
    assert bool((rest <= ref.amin(1) * (1 + 2 * unit)).all())
    assert bool(torch.isfinite(out).all())
