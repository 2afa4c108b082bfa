"""Arguments that the token and FP8 entry points refuse, before any device
call (no GPU needed)."""
import ctypes

import pytest
import torch

from moe_grouped_gemm_nvfp4_gb300 import fp8, tokens
from moe_grouped_gemm_nvfp4_gb300 import nvfp4 as F

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
HALF = ctypes.c_void_p(4104)


def test_tokens_refusals():
    lib = F.load()
    inv, uns = F.NVFP4_ERR_INVALID_ARG, F.NVFP4_ERR_UNSUPPORTED

    def dispatch(x=P, ld=64, pos=P, off=P, E=4, T=8, topk=2, R=16, D=64, dt=0, out=P):
        return lib.nvfp4_tokens_dispatch(x, ld, pos, off, E, T, topk, R, D, dt, out, None)

    def combine(y=P, ld=64, pos=P, w=P, T=8, topk=2, R=16, D=64, dt=0, out=P):
        return lib.nvfp4_tokens_combine(y, ld, pos, w, T, topk, R, D, dt, out, None)

    def grad(d=P, ld=64, y=P, ldy=64, pos=P, w=P, off=P, E=4, T=8, topk=2, R=16, D=64, dt=0, dy=P,
             dw=P):
        return lib.nvfp4_tokens_combine_grad(d, ld, y, ldy, pos, w, off, E, T, topk, R, D, dt, dy,
                                             dw, None)

    for call in (dispatch, combine, grad):
        for bad in (dict(T=-1), dict(topk=0), dict(R=-1), dict(D=0), dict(ld=63), dict(dt=3),
                    dict(dt=-1), dict(pos=None)):
            assert call(**bad) == inv, (call, bad)
        assert call(R=1 << 31) == uns
        assert call(D=(1 << 28) + 1, ld=1 << 29, **({"ldy": 1 << 29} if call is grad else {})) == uns
    assert dispatch(x=None) == inv and dispatch(out=None) == inv and dispatch(E=0) == inv
    assert combine(y=None) == inv and combine(out=None) == inv
    for name in ("d", "y", "w", "dy", "dw"):
        assert grad(**{name: None}) == inv
    assert grad(ldy=60) == inv
    assert dispatch(x=ODD) == uns and combine(out=ODD) == uns and grad(dw=ODD) == uns
    assert dispatch(x=ctypes.c_void_p(4098), dt=F.NVFP4_FP32) == uns


def test_fp8_refusals():
    lib = F.load()
    inv, uns = F.NVFP4_ERR_INVALID_ARG, F.NVFP4_ERR_UNSUPPORTED

    def quant(x=P, rows=4, cols=64, ld=64, dt=0, flags=0, pos=None, fan=1, q=P, s=P, out=4):
        return lib.nvfp4_fp8_quantize(x, rows, cols, ld, dt, flags, pos, fan, q, s, out, None)

    for bad in (dict(rows=-1), dict(cols=0), dict(ld=63), dict(dt=5), dict(flags=2), dict(fan=0),
                dict(fan=2), dict(out=5), dict(x=None), dict(q=None), dict(s=None),
                dict(flags=1, ld=64)):
        assert quant(**bad) == inv, bad
    for bad in (dict(dt=F.NVFP4_FP32), dict(cols=24, ld=24), dict(ld=68), dict(x=HALF),
                dict(q=HALF), dict(s=ODD)):
        assert quant(**bad) == uns, bad
    assert lib.nvfp4_fp8_quantize_weights(None, 1, 4, 16, 0, P, P, None) == inv
    assert lib.nvfp4_fp8_quantize_weights(P, 0, 4, 16, 0, P, P, None) == inv
    assert lib.nvfp4_fp8_quantize_weights(P, 1, 4, 24, 0, P, P, None) == uns

    def gemm(A=P, sA=P, W=P, sW=P, C=P, M=4, N=64, K=64, ldc=64, dt=0):
        return lib.nvfp4_fp8_gemm(A, sA, W, sW, C, M, N, K, ldc, dt, None)

    def grouped(A=P, sA=P, W=P, sW=P, off=P, E=4, M=4, N=64, K=64, C=P, ldc=64, dt=0):
        return lib.nvfp4_fp8_grouped_gemm(A, sA, W, sW, off, E, M, N, K, C, ldc, dt, None)

    for call in (gemm, grouped):
        for bad in (dict(A=None), dict(sA=None), dict(W=None), dict(sW=None), dict(C=None),
                    dict(M=-1), dict(N=0), dict(K=0), dict(ldc=63), dict(dt=9)):
            assert call(**bad) == inv, bad
        for bad in (dict(K=72), dict(A=HALF), dict(W=HALF), dict(C=ODD), dict(sA=ODD),
                    dict(M=(1 << 30) + 1)):
            assert call(**bad) == uns, bad
    assert grouped(off=None) == inv and grouped(E=0) == inv and grouped(E=1025) == uns


def test_python_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    pos = torch.zeros((4, 2), dtype=torch.int32)
    off = torch.zeros(5, dtype=torch.int32)
    w = torch.zeros((4, 2))
    y = torch.zeros((8, 64), dtype=torch.bfloat16)
    for bad in (pos.long(), pos[0], pos.t()):
        with pytest.raises(ValueError):
            tokens.dispatch(x, bad, off)
    with pytest.raises(ValueError):
        tokens.dispatch(x[:3], pos, off)
    with pytest.raises(ValueError):
        tokens.dispatch(x, pos, off.long())
    with pytest.raises(ValueError):
        tokens.dispatch(x.view(2, 2, 64), pos, off)
    with pytest.raises(ValueError):
        tokens.combine(y, pos, w.double())
    with pytest.raises(ValueError):
        tokens.combine(y, pos, w[:, :1])
    with pytest.raises(ValueError):
        tokens.combine_grad(x.float(), y, pos, w, off)
    with pytest.raises(ValueError):
        tokens.combine_grad(x[:, :32], y, pos, w, off)
    with pytest.raises(ValueError):                       # CPU tensors
        tokens.dispatch(x, pos, off)
    codes = torch.zeros((2, 128, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros((2, 1, 1))
    for bad_x, bad_w, bad_s in ((x, codes[0].view(torch.uint8), scales[0]), (x, codes[0], scales),
                                (x[:, :48], codes[0], scales[0]), (x.float(), codes[0], scales[0]),
                                (x, codes[0], scales[0].double()), (x, codes, scales)):
        with pytest.raises(ValueError):
            fp8.linear(bad_x, bad_w, bad_s)
    for bad_off in (off, off[:3].long(), off[:2]):
        with pytest.raises(ValueError):
            fp8.expert_linear(x, codes, scales, bad_off)
    with pytest.raises(ValueError):
        fp8.quantize_rows(x, pos[:3])
    leaf = x.clone().requires_grad_()
    with pytest.raises(RuntimeError):                     # a gradient would be lost
        fp8.linear(leaf, codes[0], scales[0])
    with pytest.raises(RuntimeError):
        fp8.expert_linear(leaf, codes, scales, off[:3])


def test_workspace_bytes():
    assert F.nvfp4_fp8_linear_workspace_bytes(5, 144) == 5 * (256 + 4 * 2)   # rows of 128 bytes
    assert F.nvfp4_fp8_linear_workspace_bytes(0, 128) == 0
    assert F.nvfp4_fp8_linear_workspace_bytes(-1, 128) == 0
    lib = F.load()
    for call, extra in ((lib.nvfp4_fp8_linear, ()), (lib.nvfp4_fp8_expert_linear, (0, None, 1))):
        middle = (P, P) if call is lib.nvfp4_fp8_linear else (P, P, P, 4, 4)
        args = (P, 4, 64, 0, *extra, *middle, 64, 64, P, 64, P)
        assert call(*args, 4 * (128 + 4) - 1, None) == F.NVFP4_ERR_UNSUPPORTED   # too small
    assert lib.nvfp4_fp8_linear(P, 4, 64, 0, P, P, 64, 64, P, 64, None, 1 << 20, None) == \
        F.NVFP4_ERR_INVALID_ARG
