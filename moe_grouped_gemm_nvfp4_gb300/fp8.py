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
from .tokens import check_routes, empty, on_stream, rows_of

BLOCK = 128


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _check_product(x, K, w, w_scale, dim):
    if w.dim() != dim or w.dtype != torch.float8_e4m3fn or not w.is_contiguous():
        raise ValueError(f"w: expected contiguous float8_e4m3fn codes of {dim} dimensions")
    shape = w.shape
    want = (*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1]))
    if w_scale.shape != want or w_scale.dtype != torch.float32 or not w_scale.is_contiguous():
        raise ValueError(f"w_scale: expected contiguous FP32 {want}")
    if K != shape[-1]:
        raise ValueError(f"x has {K} columns, the weights {shape[-1]}")
    if x.dtype != torch.bfloat16 and x.dtype != torch.float16:
        raise ValueError(f"x: expected BF16 or FP16, got {x.dtype}")


def _rows16(x, stream):
    """Rows whose base and stride are multiples of 16 bytes (a copy where not)."""
    x = rows_of(x, "x", stream)
    if x.data_ptr() % 16 or (x.shape[0] > 1 and x.stride(0) % 8):
        if stream is None:
            return x.clone(memory_format=torch.contiguous_format)
        with on_stream(stream):
            return x.clone(memory_format=torch.contiguous_format)
    return x


def _out_rows(x, route_pos, R):
    if route_pos is None:
        return x.shape[0]
    check_routes(route_pos)
    if route_pos.shape[0] != x.shape[0]:
        raise ValueError(f"{x.shape[0]} rows for the routes of {route_pos.shape[0]} tokens")
    return route_pos.numel() if R is None else R


def quantize_rows(x, route_pos=None, R=None, silu_mul: bool = False, stream=None):
    """Rows [T, K] (silu_mul: [T, 2K], quantising SiLU(first half) * second half)
    -> (codes float8_e4m3fn [R, K], scales FP32 [ceil(K/128), R]).  With
    route_pos, row t goes to the rows route_pos[t, :] (R: their number unless
    given); rows that no route names are left unwritten."""
    x = _rows16(x, stream)
    R = _out_rows(x, route_pos, R)
    K = x.shape[1] // 2 if silu_mul else x.shape[1]
    codes = empty((R, K), torch.float8_e4m3fn, x.device, stream)
    scales = empty((_blocks(K), R), torch.float32, x.device, stream)
    F.nvfp4_fp8_quantize(x, codes, scales, F.NVFP4_FP8_SILU_MUL if silu_mul else 0, route_pos,
                         stream)
    return codes, scales


def quantize_weights(w, stream=None):
    """[N, K] or [E, N, K] -> (codes, scales), one scale per 128 x 128 block."""
    w3 = (w if w.dim() == 3 else w[None]).contiguous()
    E, N, K = w3.shape
    codes = empty((E, N, K), torch.float8_e4m3fn, w.device, stream)
    scales = empty((E, _blocks(N), _blocks(K)), torch.float32, w.device, stream)
    F.nvfp4_fp8_quantize_weights(w3, codes, scales, stream)
    return (codes, scales) if w.dim() == 3 else (codes[0], scales[0])


def transpose_weights(w, w_scale):
    """Codes and scales of the transposed weights, exactly (a 128 x 128 block
    transposes into a 128 x 128 block): the product with them is the gradient
    of the activations.  N must be a multiple of 16."""
    codes = w.view(torch.uint8).transpose(-1, -2).contiguous().view(torch.float8_e4m3fn)
    return codes, w_scale.transpose(-1, -2).contiguous()


def _workspace(rows, K, device, stream):
    return empty((rows * (K + 4 * _blocks(K)),), torch.uint8, device, stream)


def linear(x, w, w_scale, stream=None):
    """y = x . w^T: x [.., K] BF16 or FP16, w codes [N, K] -> [.., N] in x's type."""
    K = x.shape[-1]
    _check_product(x, K, w, w_scale, 2)
    rows = _rows16(x if x.dim() == 2 else x.reshape(-1, K), stream)
    M, N = rows.shape[0], w.shape[0]
    y = empty((M, N), x.dtype, x.device, stream)
    F.nvfp4_fp8_linear(rows, w, w_scale, y, _workspace(M, K, x.device, stream), stream)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], N)


def expert_linear(x, w, w_scale, expert_offsets, route_pos=None, R=None, silu_mul: bool = False,
                  stream=None):
    """Each route's row times its expert's weights: w codes [E, N, K] -> [R, N]
    in expert order.  With route_pos, x is in token order and its rows are
    gathered while they are quantised; without, x is in expert order already.
    silu_mul: x holds gate and up halves [.., 2K], the rows are SiLU(gate) * up.
    Rows past expert_offsets[E] are zero."""
    K = x.shape[-1] // 2 if silu_mul else x.shape[-1]
    _check_product(x, K, w, w_scale, 3)
    if expert_offsets.dtype != torch.int32 or expert_offsets.shape != (w.shape[0] + 1,) \
            or not expert_offsets.is_contiguous():
        raise ValueError("expert_offsets: expected contiguous int32 [E + 1]")
    x = _rows16(x, stream)
    R = _out_rows(x, route_pos, R)
    y = empty((R, w.shape[1]), x.dtype, x.device, stream)
    F.nvfp4_fp8_expert_linear(x, w, w_scale, expert_offsets, y, _workspace(R, K, x.device, stream),
                              F.NVFP4_FP8_SILU_MUL if silu_mul else 0, route_pos, stream)
    return y
