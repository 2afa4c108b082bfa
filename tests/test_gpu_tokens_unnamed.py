"""Rows that no route names, without expert_offsets: they take part in the
gradients of whatever lies around dispatch and combine, so they are zero there
and hold nothing that the allocator left behind."""
import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F
from moe_grouped_gemm_nvfp4_gb300 import tokens
from test_gpu_tokens import TYPES, normal, routes

pytestmark = pytest.mark.gpu


def poison(shape, dtype):
    """Leaves blocks of this size, full of NaN, for the allocator's next calls."""
    blocks = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del blocks


def unnamed(pos, R):
    rows = torch.ones(R, dtype=torch.bool, device="cuda")
    rows[pos[pos >= 0].long()] = False
    assert rows.any()
    return rows


# aligned and odd widths; positions without a gap, a buffer that is larger
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,topk,E,D,extra", [(40, 4, 8, 256, 0), (33, 3, 5, 77, 9), (64, 8, 16, 512, 128)])
@pytest.mark.parametrize("weighted", [True, False])
def test_gradient_of_combine_without_offsets(T, topk, E, D, extra, dtype, weighted):
    pos, off = routes(T + D, T, topk, E, 0.3)
    R = T * topk + extra
    y = normal(1, (R, D), dtype).requires_grad_()
    w = torch.rand((T, topk), generator=torch.Generator().manual_seed(3)).cuda().requires_grad_() \
        if weighted else None
    c = normal(2, (T, D), dtype)
    out = tokens.combine(y, pos, w)
    poison((R, D), dtype)
    got = torch.autograd.grad(out, (y, w) if weighted else (y,), c)
    dead = unnamed(pos, R)
    assert torch.equal(got[0][dead], torch.zeros_like(got[0][dead]))
    want = torch.autograd.grad(tokens.combine(y, pos, w, off), (y, w) if weighted else (y,), c)
    assert torch.equal(got[0][~dead], want[0][~dead])
    if weighted:
        assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("leaf", ["tokens", "weights"])
def test_experts_weight_gradient_through_rows_of_no_route(dtype, leaf):
    """dW = rows^T dy sums over every row of the buffer."""
    T, topk, E, D, N = 48, 4, 8, 128, 64
    pos, off = routes(9, T, topk, E, 0.3)
    x = normal(1, (T, D), dtype)
    if leaf == "tokens":
        x.requires_grad_()
    m = (normal(2, (D, N), dtype) * D ** -0.5).requires_grad_()
    c = normal(3, (T, N), dtype)

    def grads(*offsets):
        poison((T * topk, D), dtype)
        rows = tokens.dispatch(x, pos, *offsets)
        y = rows @ m
        poison((T * topk, N), dtype)
        return rows, *torch.autograd.grad(tokens.combine(y, pos, None, *offsets), m, c)

    rows, got = grads()
    rows_off, want = grads(off)
    assert torch.equal(rows, rows_off)
    assert torch.equal(got, want)


def test_filling_is_captured_and_no_grad_keeps_its_values():
    T, topk, E, D = 32, 4, 8, 96
    pos, off = routes(4, T, topk, E, 0.3)
    x = normal(1, (T, D), torch.bfloat16)
    want = tokens.dispatch(x, pos, off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows = tokens.dispatch(x, pos)
    rows.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(rows, want)
    with torch.no_grad():
        named = ~unnamed(pos, T * topk)
        assert torch.equal(tokens.dispatch(x, pos)[named], want[named])
    assert F.nvfp4_device_status() == F.NVFP4_OK
