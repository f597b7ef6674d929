"""FP8 E4M3 in blocks of 128: RMSNorm with a block-quantised output, quantising a matrix, and
the product of two block-scaled matrices (through the native binding; the contracts stand in
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

from . import _check, lib
from ._launch import native, on_stream

_vp, _f32, _i64, _int = ctypes.c_void_p, ctypes.c_float, ctypes.c_int64, ctypes.c_int
lib.fused_add_rmsnorm_quant_block.argtypes = [_vp, _i64, _vp, _i64, _vp, _f32, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp]
lib.fused_add_rmsnorm_quant_block.restype = _int
lib.rmsnorm_quant_block.argtypes = [_vp, _i64, _vp, _f32, _vp, _vp, _i64, _i64, _int, _vp]
lib.rmsnorm_quant_block.restype = _int
lib.quant_block_fp8.argtypes = [_vp, _i64, _vp, _vp, _i64, _i64, _int, _int, _int, _vp]
lib.quant_block_fp8.restype = _int
lib.gemm_fp8_block.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _int, _vp, _i64, _i64, _i64, _i64, _int, _vp]
lib.gemm_fp8_block.restype = _int
lib.far_plan_gemm_fp8_for_sms.argtypes = [_i64, _i64, _i64, _int, _int, _vp]
lib.far_plan_gemm_fp8_for_sms.restype = _int

BLOCKS = {"row": 0, "tile": 1}


def fused_add_rmsnorm_quant_block(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, eps: float,
                                  q: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                                  residual_out: torch.Tensor | None = None, stream=None):
    """(q, scale, residual_out): fused_add_rmsnorm with its output in E4M3 blocks of 128.

    q is [..., hidden] float8_e4m3fn, scale [..., ceil(hidden / 128)] float32; a block
    dequantises as q * scale.  Pass residual_out=residual for in-place use.
    """
    if residual is None:
        raise ValueError("residual is missing: rmsnorm_quant_block takes x alone")
    if stream is None:
        return native.norm_quant_block(x, residual, weight, eps, q, scale, residual_out)
    return on_stream(stream, native.norm_quant_block, x, residual, weight, eps, q, scale, residual_out)


def rmsnorm_quant_block(x: torch.Tensor, weight: torch.Tensor, eps: float, q: torch.Tensor | None = None,
                        scale: torch.Tensor | None = None, stream=None):
    """(q, scale): rmsnorm with its output in E4M3 blocks of 128."""
    if stream is None:
        return native.norm_quant_block(x, None, weight, eps, q, scale, None)
    return on_stream(stream, native.norm_quant_block, x, None, weight, eps, q, scale, None)


def quant_block_fp8(x: torch.Tensor, block: str = "row", transpose: bool = False, q: torch.Tensor | None = None,
                    scale: torch.Tensor | None = None, stream=None):
    """(q, scale): a 2-D float32, float16 or bfloat16 matrix in E4M3 blocks of 128.

    block "row": a scale for each 128 values of a row of q; "tile": for each 128 x 128 tile.
    transpose=True writes q as x's transpose ([cols, rows], contiguous).
    """
    if block not in BLOCKS:
        raise ValueError('block is "row" or "tile"')
    if stream is None:
        return native.quant_block_fp8(x, BLOCKS[block], bool(transpose), q, scale)
    return on_stream(stream, native.quant_block_fp8, x, BLOCKS[block], bool(transpose), q, scale)


def gemm_fp8_block(x: torch.Tensor, x_scale: torch.Tensor, wt: torch.Tensor, wt_scale: torch.Tensor,
                   out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None, stream=None):
    """out = (x * x_scale) @ (wt * wt_scale)^T of E4M3 matrices scaled in blocks of 128 along k.

    x: [..., k], x_scale: [..., ceil(k/128)]; wt: [n, k]; wt_scale: [ceil(n/128), ceil(k/128)]
    (tiles) or [n, ceil(k/128)] (rows).  Accumulation is float32; one rounding to out_dtype.
    """
    if stream is None:
        return native.gemm_fp8_block(x, x_scale, wt, wt_scale, out_dtype, out)
    return on_stream(stream, native.gemm_fp8_block, x, x_scale, wt, wt_scale, out_dtype, out)


def plan_gemm_fp8_for_sms(m: int, n: int, k: int, block: str, sms: int) -> dict:
    """gemm_fp8_block's plan for aligned operands on a device with `sms` SMs (host logic only)."""
    buf = (ctypes.c_int * 4)()
    _check(lib.far_plan_gemm_fp8_for_sms(m, n, k, BLOCKS[block], sms, ctypes.addressof(buf)))
    return dict(zip(("kind", "rows", "split", "grid"), list(buf)))
