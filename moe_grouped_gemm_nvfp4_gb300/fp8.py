"""Products with 8-bit (E4M3) weights: one FP32 scale per 128 x 128 block of
the weights and per 1 x 128 block of the activations, dense or grouped by
expert.

Weights are codes [N, K] (or [E, N, K]) and scales [ceil(N/128), ceil(K/128)]
(or [E, ..]), as checkpoints hold them; `quantize_weights` makes them.
Activations are BF16 or FP16 rows, quantised inside `linear` and
`expert_linear`.  The gradient of the activations is the same product with the
weights transposed (`transpose_weights`, prepared once); the weights themselves
are frozen.  The quantisers round and have no derivative; the products refuse
tensors that would lose one.

Work goes to the current stream of the tensors' device, whichever device is
current, or to `stream` (a torch stream of that device or a raw handle), where
outputs and workspace are then allocated too.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import nvfp4 as F
from .nvfp4 import native
from .tokens import on_stream, refuse_tangents

BLOCK = 128


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def quantize_rows(x, route_pos=None, R=None, silu_mul: bool = False, stream=None):
    """Rows [T, K] (silu_mul: [T, 2K], quantising SiLU(first half) * second half)
    -> (codes float8_e4m3fn [R, K], scales FP32 [ceil(K/128), R]).  With
    route_pos, row t goes to the rows route_pos[t, :] (R: their number unless
    given); rows that no route names are left unwritten."""
    if stream is not None:
        with on_stream(stream, x.device):
            return quantize_rows(x, route_pos, R, silu_mul)
    if x.dim() != 2 or x.shape[1] == 0 or (silu_mul and x.shape[1] % 2):
        raise ValueError(f"x: expected rows, got shape {tuple(x.shape)}")
    T, width = x.shape
    if route_pos is None:
        R = T
    else:
        if route_pos.dim() != 2 or route_pos.dtype != torch.int32 \
                or not route_pos.is_contiguous() or route_pos.shape[0] != T:
            raise ValueError("route_pos: expected contiguous int32 [T, topk]")
        if route_pos.device != x.device:
            raise ValueError("tensors on different devices")
        R = route_pos.numel() if R is None else R
    if x.stride(1) != 1 or (T > 1 and (x.stride(0) < width or x.stride(0) % 8)) \
            or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)
    K = width // 2 if silu_mul else width
    codes = torch.empty((R, K), dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((_blocks(K), R), dtype=torch.float32, device=x.device)
    with torch.cuda.device_of(x):
        F.nvfp4_fp8_quantize(x, codes, scales, F.NVFP4_FP8_SILU_MUL if silu_mul else 0, route_pos)
    return codes, scales


def quantize_weights(w, stream=None):
    """[N, K] or [E, N, K] -> (codes, scales), one scale per 128 x 128 block."""
    if stream is not None:
        with on_stream(stream, w.device):
            return quantize_weights(w)
    w3 = (w if w.dim() == 3 else w[None]).contiguous()
    E, N, K = w3.shape
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=w.device)
    scales = torch.empty((E, _blocks(N), _blocks(K)), dtype=torch.float32, device=w.device)
    with torch.cuda.device_of(w3):
        F.nvfp4_fp8_quantize_weights(w3, codes, scales)
    return (codes, scales) if w.dim() == 3 else (codes[0], scales[0])


def transpose_weights(w, w_scale):
    """Codes and scales of the transposed weights, exactly (a 128 x 128 block
    transposes into a 128 x 128 block): the product with them is the gradient
    of the activations.  N must be a multiple of 16."""
    codes = w.view(torch.uint8).transpose(-1, -2).contiguous().view(torch.float8_e4m3fn)
    return codes, w_scale.transpose(-1, -2).contiguous()


def linear(x, w, w_scale, stream=None):
    """y = x . w^T: x [.., K] BF16 or FP16, w codes [N, K] -> [.., N] in x's type."""
    if forward_ad._current_level >= 0:
        refuse_tangents(x, w, w_scale)
    if stream is not None:
        with on_stream(stream, x.device):
            return linear(x, w, w_scale)
    if x.dim() == 2:
        return native().linear(x, w, w_scale)
    y = native().linear(x.reshape(-1, x.shape[-1]), w, w_scale)
    return y.view(*x.shape[:-1], y.shape[1])


def linear_codes(codes, scales, w, w_scale, dtype=torch.bfloat16, stream=None):
    """y = x . w^T for rows that are quantised already (quantize_rows,
    norm.rms_norm_fp8): codes float8_e4m3fn [M, K], scales FP32 [ceil(K / 128), M], w
    codes [N, K] -> [M, N] of `dtype` (BF16, FP16 or FP32)."""
    if forward_ad._current_level >= 0:
        refuse_tangents(scales, w_scale)
    if dtype not in F._DTYPES:
        raise ValueError(f"dtype: expected BF16, FP16 or FP32, got {dtype}")
    if stream is not None:
        with on_stream(stream, codes.device):
            return native().linear_codes(codes, scales, w, w_scale, F._DTYPES[dtype])
    return native().linear_codes(codes, scales, w, w_scale, F._DTYPES[dtype])


def expert_linear(x, w, w_scale, expert_offsets, route_pos=None, R=None, silu_mul: bool = False,
                  stream=None):
    """Each route's row times its expert's weights: w codes [E, N, K] -> [R, N]
    in expert order.  With route_pos, x is in token order and its rows are
    gathered while they are quantised (R: the routes' number unless given);
    without, x is in expert order already.  silu_mul: x holds gate and up halves
    [.., 2K], the rows are SiLU(gate) * up.  Rows past expert_offsets[E] are
    zero."""
    if forward_ad._current_level >= 0:
        refuse_tangents(x, w, w_scale)
    R = -1 if R is None else R
    if stream is not None:
        with on_stream(stream, x.device):
            return native().expert_linear(x, w, w_scale, expert_offsets, route_pos, R, silu_mul)
    return native().expert_linear(x, w, w_scale, expert_offsets, route_pos, R, silu_mul)
