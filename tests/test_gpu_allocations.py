"""Outputs of the native calls are allocated where torch's own modes see them: dispatch modes, and
the fill of uninitialised memory that deterministic algorithms ask for."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from moe_grouped_gemm_nvfp4_gb300 import gating, norm, tokens

pytestmark = pytest.mark.gpu


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.names = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.names.append(str(func))
        return func(*args, **(kwargs or {}))


def test_dispatch_modes_see_the_outputs():
    x = torch.randn((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1)
    with torch.no_grad():
        for call, outputs in ((lambda: norm.rms_norm(x, w, x), 2), (lambda: gating.topk_gate(x, 2), 2),
                              (lambda: tokens.dispatch(x, pos), 1), (lambda: tokens.combine(x, pos), 1)):
            plain = call()
            with Seen() as seen:
                got = call()
            assert sum(n.startswith("aten.empty") for n in seen.names) == outputs, seen.names
            for a, b in zip(plain if isinstance(plain, tuple) else (plain,),
                            got if isinstance(got, tuple) else (got,)):
                assert torch.equal(a, b)


def test_deterministic_fill_reaches_rows_that_no_route_names():
    x = torch.randn((4, 64), device="cuda").bfloat16()
    pos = torch.tensor([[0], [2], [4], [6]], dtype=torch.int32, device="cuda")
    before = torch.are_deterministic_algorithms_enabled()
    fill = torch.utils.deterministic.fill_uninitialized_memory
    try:
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = True
        with torch.no_grad():
            out = tokens.dispatch(x, pos, R=8)
    finally:
        torch.use_deterministic_algorithms(before)
        torch.utils.deterministic.fill_uninitialized_memory = fill
    assert torch.equal(out[::2], x)
    assert bool(torch.isnan(out[1::2]).all())
