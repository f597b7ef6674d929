"""The gated feed-forward block's way in, and its gradients (through the native binding; the contracts
stand in ``include/far.h`` at gated_ffn and gated_ffn_backward).

    h = gated_ffn(x, w_gate, w_up)                                          # act(x @ w_gate^T) * (x @ w_up^T)

Training keeps both projections for the way back:

    h, gate, up = gated_ffn(x, w_gate, w_up, save=True)
    dx, dw_gate, dw_up = gated_ffn_backward(dh, gate, up, x, w_gate, w_up)

Serving in 8 bits behind it: ``gemm_int8(*quant_rows_int8(h), down_q, down_scale)``.
"""
from __future__ import annotations

import ctypes

import torch

from . import FarError, _check, lib
from ._launch import native, on_stream

_vp, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_MATRIX = [_vp, _i64]
lib.gated_ffn.argtypes = _MATRIX * 6 + [_i64, _i64, _i64, _int, _int, _vp]
lib.gated_ffn.restype = _int
lib.far_gated_ffn_backward_workspace_bytes.argtypes = [_i64, _i64]
lib.far_gated_ffn_backward_workspace_bytes.restype = _i64
lib.gated_ffn_backward.argtypes = _MATRIX * 9 + [_vp, _i64, _i64, _i64, _i64, _int, _int, _vp]
lib.gated_ffn_backward.restype = _int
lib.far_plan_gated_ffn.argtypes = [_i64, _i64, _i64, _vp]
lib.far_plan_gated_ffn.restype = _int

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def _code(activation: str) -> int:
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[activation]


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu", save: bool = False,
              out: torch.Tensor | None = None, gate_out: torch.Tensor | None = None, up_out: torch.Tensor | None = None,
              stream=None):
    """act(x @ w_gate^T) * (x @ w_up^T), or with save=True (that, x @ w_gate^T, x @ w_up^T).

    x: [..., tokens, hidden], w_gate and w_up: [ffn, hidden], all float16 or all bfloat16.  The projections
    stay in float32 until the product; the kept ones are rounded.
    """
    if not save and (gate_out is not None or up_out is not None):
        raise ValueError("gate_out and up_out are written with save=True")
    args = (x, w_gate, w_up, _code(activation), bool(save), out, gate_out, up_out)
    return native.gated_ffn(*args) if stream is None else on_stream(stream, native.gated_ffn, *args)


def gated_ffn_backward_workspace_bytes(tokens: int, ffn: int) -> int:
    n = lib.far_gated_ffn_backward_workspace_bytes(tokens, ffn)
    if n < 0:
        raise FarError(-n)
    return n


def gated_ffn_backward(dout: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor,
                       w_up: torch.Tensor, activation: str = "silu", dx: torch.Tensor | None = None,
                       dw_gate: torch.Tensor | None = None, dw_up: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None):
    """(dx, dw_gate, dw_up): gated_ffn's gradients given its output's, at the projections it kept.

    Sums over tokens are float32, in a fixed order; the gradients have the inputs' dtype.  What the sums are
    of, the projections' gradients, is rounded to that dtype first (float16: infinite from 65520 up).
    workspace: gated_ffn_backward_workspace_bytes(tokens, ffn) bytes, allocated when not given; calls
    that may overlap need one each.
    """
    args = (dout, gate, up, x, w_gate, w_up, _code(activation), dx, dw_gate, dw_up, workspace)
    return native.gated_ffn_backward(*args) if stream is None else on_stream(stream, native.gated_ffn_backward, *args)


def plan_gated_ffn(tokens: int, hidden: int, ffn: int) -> dict:
    """gated_ffn's plan for aligned operands (host logic only)."""
    buf = (ctypes.c_int * 3)()
    _check(lib.far_plan_gated_ffn(tokens, hidden, ffn, ctypes.addressof(buf)))
    return dict(zip(("kind", "tokens", "split"), list(buf)))
