"""Products with 8-bit (E4M3) weights: one FP32 scale per 128 x 128 block of
the weights and per 1 x 128 block of the activations, dense or grouped by
expert.

Weights are codes [N, K] (or [E, N, K]) and scales [ceil(N/128), ceil(K/128)]
(or [E, ..]), as checkpoints hold them; `quantize_weights` makes them.
Activations are BF16 or FP16 rows, quantised inside `linear` and
`expert_linear`.  The gradient of the activations is the same product with the
weights transposed (`transpose_weights`, prepared once); the weights themselves
are frozen.
"""
from __future__ import annotations

import torch

from . import nvfp4 as F
from .tokens import check_routes, on_stream, rows_of

BLOCK = 128


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _check_product(x, w, w_scale, dim):
    if w.dim() != dim or w.dtype != torch.float8_e4m3fn or not w.is_contiguous():
        raise ValueError(f"w: expected contiguous float8_e4m3fn codes of {dim} dimensions")
    want = (*w.shape[:-2], _blocks(w.shape[-2]), _blocks(w.shape[-1]))
    if tuple(w_scale.shape) != want or w_scale.dtype != torch.float32 \
            or not w_scale.is_contiguous():
        raise ValueError(f"w_scale: expected contiguous FP32 {want}")
    if x.shape[-1] != w.shape[-1]:
        raise ValueError(f"x has {x.shape[-1]} columns, the weights {w.shape[-1]}")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"x: expected BF16 or FP16, got {x.dtype}")


def quantize_rows(x, route_pos=None, R=None, silu_mul: bool = False, stream=None):
    """Rows [T, K] (silu_mul: [T, 2K], quantising SiLU(first half) * second half)
    -> (codes float8_e4m3fn [R, K], scales FP32 [ceil(K/128), R]).  With
    route_pos, row t goes to the rows route_pos[t, :] (R: their number unless
    given); rows that no route names are left unwritten."""
    x = rows_of(x, "x")
    if route_pos is not None:
        check_routes(route_pos)
        if route_pos.shape[0] != x.shape[0]:
            raise ValueError(f"{x.shape[0]} rows for the routes of {route_pos.shape[0]} tokens")
        R = route_pos.numel() if R is None else R
    else:
        R = x.shape[0]
    K = x.shape[1] // 2 if silu_mul else x.shape[1]
    with on_stream(stream):
        if x.data_ptr() % 16 or (x.shape[0] > 1 and x.stride(0) % 8):
            x = x.clone(memory_format=torch.contiguous_format)
        codes = torch.empty((R, K), dtype=torch.float8_e4m3fn, device=x.device)
        scales = torch.empty((_blocks(K), R), dtype=torch.float32, device=x.device)
    F.nvfp4_fp8_quantize(x, codes, scales, F.NVFP4_FP8_SILU_MUL if silu_mul else 0, route_pos,
                         stream)
    return codes, scales


def quantize_weights(w, stream=None):
    """[N, K] or [E, N, K] -> (codes, scales), one scale per 128 x 128 block."""
    w3 = (w if w.dim() == 3 else w[None]).contiguous()
    E, N, K = w3.shape
    with on_stream(stream):
        codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=w.device)
        scales = torch.empty((E, _blocks(N), _blocks(K)), dtype=torch.float32, device=w.device)
    F.nvfp4_fp8_quantize_weights(w3, codes, scales, stream)
    return (codes, scales) if w.dim() == 3 else (codes[0], scales[0])


def transpose_weights(w, w_scale):
    """Codes and scales of the transposed weights, exactly (a 128 x 128 block
    transposes into a 128 x 128 block): the product with them is the gradient
    of the activations.  N must be a multiple of 16."""
    codes = w.view(torch.uint8).transpose(-1, -2).contiguous().view(torch.float8_e4m3fn)
    return codes, w_scale.transpose(-1, -2).contiguous()


def linear(x, w, w_scale, stream=None):
    """y = x . w^T: x [.., K] BF16 or FP16, w codes [N, K] -> [.., N] in x's type."""
    _check_product(x, w, w_scale, 2)
    rows = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    codes, scales = quantize_rows(rows, stream=stream)
    with on_stream(stream):
        y = torch.empty((rows.shape[0], w.shape[0]), dtype=x.dtype, device=x.device)
    F.nvfp4_fp8_gemm(codes, scales, w, w_scale, y, stream)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], w.shape[0])


def expert_linear(x, w, w_scale, expert_offsets, route_pos=None, R=None, silu_mul: bool = False,
                  stream=None):
    """Each route's row times its expert's weights: w codes [E, N, K] -> [R, N]
    in expert order.  With route_pos, x is in token order and its rows are
    gathered while they are quantised; without, x is in expert order already.
    silu_mul: x holds gate and up halves [.., 2K], the rows are SiLU(gate) * up.
    Rows past expert_offsets[E] are zero."""
    _check_product(x[:, :x.shape[1] // 2] if silu_mul else x, w, w_scale, 3)
    if expert_offsets.dtype != torch.int32 or expert_offsets.shape != (w.shape[0] + 1,) \
            or not expert_offsets.is_contiguous():
        raise ValueError("expert_offsets: expected contiguous int32 [E + 1]")
    codes, scales = quantize_rows(x, route_pos, R, silu_mul, stream)
    with on_stream(stream):
        y = torch.empty((codes.shape[0], w.shape[1]), dtype=x.dtype, device=x.device)
    F.nvfp4_fp8_grouped_gemm(codes, scales, w, w_scale, expert_offsets, y, stream)
    return y
