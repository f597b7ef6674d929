"""FP8 E4M3 in blocks of 128: RMSNorm with a block-quantised output, quantising a matrix, and
the product of two block-scaled matrices (ctypes binding; the contracts stand in
``include/far.h`` at fused_add_rmsnorm_quant_block, quant_block_fp8 and gemm_fp8_block).

    wq, ws = quant_block_fp8(weight, block="tile")                     # once
    xq, xs, residual = fused_add_rmsnorm_quant_block(x, residual, norm_weight, 1e-6)
    y = gemm_fp8_block(xq, xs, wq, ws)                                 # y = norm(x + residual) @ weight^T

Training: with y = x @ w^T and dy its gradient, dx takes dy by rows and w transposed by tiles,
dw takes dy and x transposed by rows (the sum runs over the tokens):

    dx = gemm_fp8_block(*quant_block_fp8(dy), *quant_block_fp8(w, block="tile", transpose=True))
    dw = gemm_fp8_block(*quant_block_fp8(dy, transpose=True), *quant_block_fp8(x, transpose=True),
                        out_dtype=torch.float32)
"""
from __future__ import annotations

import ctypes

import torch

from . import TORCH_TO_CODE, FarError, _row_stride, dtypes, lib
from ._launch import Launch, ptr

_vp, _f32, _i64, _int = ctypes.c_void_p, ctypes.c_float, ctypes.c_int64, ctypes.c_int
lib.fused_add_rmsnorm_quant_block.argtypes = [_vp, _i64, _vp, _i64, _vp, _f32, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp]
lib.fused_add_rmsnorm_quant_block.restype = _int
lib.rmsnorm_quant_block.argtypes = [_vp, _i64, _vp, _f32, _vp, _vp, _i64, _i64, _int, _vp]
lib.rmsnorm_quant_block.restype = _int
lib.quant_block_fp8.argtypes = [_vp, _i64, _vp, _vp, _i64, _i64, _int, _int, _int, _vp]
lib.quant_block_fp8.restype = _int
lib.gemm_fp8_block.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _int, _vp, _i64, _i64, _i64, _i64, _int, _vp]
lib.gemm_fp8_block.restype = _int

E4M3 = torch.float8_e4m3fn
BLOCKS = {"row": 0, "tile": 1}


def _blocks(n: int) -> int:
    return (n + 127) >> 7


def _rows_of(t: torch.Tensor):
    """(rows, values a row, row stride) of a [..., n] tensor whose rows are evenly spaced."""
    if t.is_contiguous():
        n = t.shape[-1]
        return (t.numel() // n if n else 0), n, n
    st = _row_stride(t)
    if st is None:
        raise ValueError("non-contiguous tensors must be 2-D with contiguous rows")
    return t.shape[0], t.shape[1], st


def _codes(go, q, shape):
    if q is None:
        return go.empty(shape, E4M3)
    if tuple(q.shape) != tuple(shape) or q.dtype not in (E4M3, torch.uint8) or not q.is_contiguous():
        raise ValueError("q must be a contiguous float8_e4m3fn (or uint8) tensor of the output's shape")
    return q


def _scales(go, scale, shape):
    if scale is None:
        return go.empty(shape, torch.float32)
    if tuple(scale.shape) != tuple(shape) or scale.dtype != torch.float32 or not scale.is_contiguous():
        raise ValueError("scale must be a contiguous float32 tensor, one value a block")
    return scale


def _norm_weight(x, weight):
    if not weight.is_contiguous() or weight.numel() != x.shape[-1]:
        raise ValueError("weight must be a contiguous [hidden] tensor")
    return dtypes(x.dtype, weight.dtype)


def fused_add_rmsnorm_quant_block(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, eps: float,
                                  q: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                                  residual_out: torch.Tensor | None = None, stream=None):
    """(q, scale, residual_out): fused_add_rmsnorm with its output in E4M3 blocks of 128.

    q is [..., hidden] float8_e4m3fn, scale [..., ceil(hidden / 128)] float32; a block
    dequantises as q * scale.  Pass residual_out=residual for in-place use.
    """
    code = _norm_weight(x, weight)
    if residual.shape != x.shape or residual.dtype != x.dtype:
        raise ValueError("x and residual must share a shape and a dtype")
    go = Launch(stream, x, residual, weight, q, scale, residual_out)
    if residual_out is None:
        residual_out = go.empty(x.shape, x.dtype)
    elif residual_out.shape != x.shape or residual_out.dtype != x.dtype:
        raise ValueError("residual_out has x's shape and dtype")
    q = _codes(go, q, x.shape)
    scale = _scales(go, scale, (*x.shape[:-1], _blocks(x.shape[-1])))
    rows, hidden, sx = _rows_of(x)
    go.run(lib.fused_add_rmsnorm_quant_block, ptr(x), sx, ptr(residual), _rows_of(residual)[2], ptr(weight), eps, ptr(q),
           ptr(scale), ptr(residual_out), _rows_of(residual_out)[2], rows, hidden, code)
    return q, scale, residual_out


def rmsnorm_quant_block(x: torch.Tensor, weight: torch.Tensor, eps: float, q: torch.Tensor | None = None,
                        scale: torch.Tensor | None = None, stream=None):
    """(q, scale): rmsnorm with its output in E4M3 blocks of 128."""
    code = _norm_weight(x, weight)
    go = Launch(stream, x, weight, q, scale)
    q = _codes(go, q, x.shape)
    scale = _scales(go, scale, (*x.shape[:-1], _blocks(x.shape[-1])))
    rows, hidden, sx = _rows_of(x)
    go.run(lib.rmsnorm_quant_block, ptr(x), sx, ptr(weight), eps, ptr(q), ptr(scale), rows, hidden, code)
    return q, scale


def quant_block_fp8(x: torch.Tensor, block: str = "row", transpose: bool = False, q: torch.Tensor | None = None,
                    scale: torch.Tensor | None = None, stream=None):
    """(q, scale): a 2-D float32, float16 or bfloat16 matrix in E4M3 blocks of 128.

    block "row": a scale for each 128 values of a row of q; "tile": for each 128 x 128 tile.
    transpose=True writes q as x's transpose ([cols, rows], contiguous).
    """
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    if block not in BLOCKS:
        raise ValueError('block is "row" or "tile"')
    if x.dtype not in TORCH_TO_CODE:
        raise FarError(2)
    go = Launch(stream, x, q, scale)
    rows, cols = x.shape
    st = _row_stride(x)
    if st is None:
        raise ValueError("x must have contiguous rows")
    r, c = (cols, rows) if transpose else (rows, cols)
    q = _codes(go, q, (r, c))
    scale = _scales(go, scale, (r if block == "row" else _blocks(r), _blocks(c)))
    go.run(lib.quant_block_fp8, ptr(x), st, ptr(q), ptr(scale), rows, cols, BLOCKS[block], int(transpose),
           TORCH_TO_CODE[x.dtype])
    return q, scale


def gemm_fp8_block(x: torch.Tensor, x_scale: torch.Tensor, wt: torch.Tensor, wt_scale: torch.Tensor,
                   out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None, stream=None):
    """out = (x * x_scale) @ (wt * wt_scale)^T of E4M3 matrices scaled in blocks of 128 along k.

    x: [..., k], x_scale: [..., ceil(k/128)]; wt: [n, k]; wt_scale: [ceil(n/128), ceil(k/128)]
    (tiles) or [n, ceil(k/128)] (rows).  Accumulation is float32; one rounding to out_dtype.
    """
    if x.dtype not in (E4M3, torch.uint8) or wt.dtype not in (E4M3, torch.uint8):
        raise ValueError("x and wt hold E4M3 codes (float8_e4m3fn or uint8)")
    if x.dim() < 2 or wt.dim() != 2 or x.shape[-1] != wt.shape[1]:
        raise ValueError("x is [..., k] and wt [n, k]")
    n, k = wt.shape
    kb = _blocks(k)
    lead = x.shape[:-1]
    if out_dtype not in TORCH_TO_CODE:
        raise FarError(2)
    if x_scale.shape != (*lead, kb) or x_scale.dtype != torch.float32 or not x_scale.is_contiguous():
        raise ValueError("x_scale must be a contiguous float32 [..., ceil(k / 128)] tensor")
    if wt_scale.dtype != torch.float32 or not wt_scale.is_contiguous() or wt_scale.dim() != 2 or wt_scale.shape[1] != kb:
        raise ValueError("wt_scale must be a contiguous float32 [.., ceil(k / 128)] tensor")
    tiles = _blocks(n)
    if wt_scale.shape[0] not in (tiles, n):
        raise ValueError("wt_scale has one row for each 128 rows of wt, or one for each")
    # (n = 1 has one of either: the same numbers)
    block = BLOCKS["tile"] if wt_scale.shape[0] == tiles else BLOCKS["row"]
    go = Launch(stream, x, x_scale, wt, wt_scale, out)
    if out is None:
        out = go.empty((*lead, n), out_dtype)
    elif out.shape != (*lead, n) or out.dtype != out_dtype:
        raise ValueError("out has shape [..., n] and out_dtype")
    m = x.numel() // k if k else out.numel() // n if n else 0
    sx = _rows_of(x)[2] if k else 0
    sw = _rows_of(wt)[2] if k else 0
    go.run(lib.gemm_fp8_block, ptr(x), sx, ptr(x_scale), ptr(wt), sw, ptr(wt_scale), block, ptr(out), _rows_of(out)[2], m, n,
           k, TORCH_TO_CODE[out_dtype])
    return out
