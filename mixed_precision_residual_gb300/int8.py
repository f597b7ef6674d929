"""int8 with a scale for each row: quantising a matrix, and the product of two such matrices (through
the native binding; the contracts stand in ``include/far.h`` at quant_rows_int8 and gemm_int8).

    wq, ws = quant_rows_int8(weight)                                              # once: a scale a channel
    xq, xs, residual = fused_add_rmsnorm_quant(x, residual, norm_weight, 1e-6, "int8")
    y = gemm_int8(xq, xs, wq, ws, bias)                        # y = norm(x + residual) @ weight^T + bias
"""
from __future__ import annotations

import ctypes

import torch

from . import FarError, _check, lib
from ._launch import native, on_stream

_vp, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
lib.quant_rows_int8.argtypes = [_vp, _i64, _vp, _vp, _i64, _i64, _int, _vp]
lib.quant_rows_int8.restype = _int
lib.far_gemm_int8_workspace_bytes.argtypes = [_i64, _i64, _i64]
lib.far_gemm_int8_workspace_bytes.restype = _i64
lib.gemm_int8.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _int, _vp]
lib.gemm_int8.restype = _int
lib.far_plan_gemm_int8.argtypes = [_i64, _i64, _i64, _vp]
lib.far_plan_gemm_int8.restype = _int


def quant_rows_int8(x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """(q, scale): the rows of a float32, float16 or bfloat16 tensor [..., cols] in int8, scale [...] float32.

    A row dequantises as q * scale: a weight's output channels, or activations' tokens (what
    fused_add_rmsnorm_quant gives of the norm's output).
    """
    if stream is None:
        return native.quant_rows_int8(x, q, scale)
    return on_stream(stream, native.quant_rows_int8, x, q, scale)


def gemm_int8_workspace_bytes(m: int, n: int, k: int) -> int:
    b = lib.far_gemm_int8_workspace_bytes(m, n, k)
    if b < 0:
        raise FarError(-b)
    return b


def gemm_int8(x: torch.Tensor, x_scale: torch.Tensor, wt: torch.Tensor, wt_scale: torch.Tensor,
              bias: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None):
    """out = (x * x_scale) @ (wt * wt_scale)^T + bias of int8 matrices with a scale for each row.

    x: [..., k], x_scale: [...]; wt: [n, k], wt_scale: [n]; bias: [n] of out_dtype; out: [..., n].  One
    token's vector has a scale without an axis, as quant_rows_int8 gives it.  The integer sums are
    exact (k <= 131071); one rounding to out_dtype behind the scales and the bias.
    workspace: gemm_int8_workspace_bytes(m, n, k) bytes, allocated when not given; calls that may
    overlap need one each.
    """
    args = (x, x_scale, wt, wt_scale, bias, out_dtype, out, workspace)
    return native.gemm_int8(*args) if stream is None else on_stream(stream, native.gemm_int8, *args)


def plan_gemm_int8(m: int, n: int, k: int) -> dict:
    """gemm_int8's plan for aligned operands (host logic only)."""
    buf = (ctypes.c_int * 3)()
    _check(lib.far_plan_gemm_int8(m, n, k, ctypes.addressof(buf)))
    return dict(zip(("kind", "rows", "split"), list(buf)))
