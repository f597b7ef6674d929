"""Per-head RMSNorm of queries and keys with the rotation by position, its gradients, the
rotation alone, and the table of cosines and sines they read (tensor calls through the native
binding, frequencies and tables through ctypes; the contract stands in ``include/far.h`` at
qk_norm_rope).

    table = rope_table(32768, 128, base=1e6, scaling={"type": "yarn", "factor": 4.0, "trained": 8192})
    q, k = qk_norm_rope(q, k, q_weight, k_weight, 1e-6, table, positions)
    dq, dk, dq_weight, dk_weight = qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, 1e-6, table, positions)

q and k are [tokens, heads, head_dim] (or [..., heads, head_dim] where the leading axes
collapse to one stride), with any strides as long as a head's values are contiguous: views
of a packed projection, and head-major [heads, tokens, head_dim] buffers transposed, are
taken as they are.  k may be None (queries alone).
"""
from __future__ import annotations

import ctypes

import torch

from . import FarError, _check, lib
from ._launch import native, on_stream

_vp, _i64, _int, _f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
_f32 = ctypes.c_float
_HEADS = [_vp, _i64, _i64]
_PLACE = [_vp, _i64, _vp, _int]  # table, rows, positions, bytes a position
_SIZES = [_i64] * 5
lib.qk_norm_rope.argtypes = _HEADS * 2 + [_vp, _vp, _f32] + _PLACE + _HEADS * 2 + _SIZES + [_int, _int, _vp]
lib.qk_norm_rope.restype = _int
lib.rope.argtypes = _HEADS * 2 + _PLACE + _HEADS * 2 + _SIZES + [_int, _int, _int, _vp]
lib.rope.restype = _int
lib.qk_norm_rope_backward.argtypes = (_HEADS * 4 + [_vp, _vp, _f32] + _PLACE + _HEADS * 2 + [_vp, _vp, _vp, _i64] +
                                      _SIZES + [_int, _int, _vp])
lib.qk_norm_rope_backward.restype = _int
lib.far_qk_backward_workspace_bytes.argtypes = [_i64]
lib.far_qk_backward_workspace_bytes.restype = _i64
lib.far_rope_frequencies.argtypes = [_i64, _f64, _int, _vp, _vp, _vp]
lib.far_rope_frequencies.restype = _int
lib.rope_table.argtypes = [_vp, _i64, _i64, _i64, _vp, _f64, _vp]
lib.rope_table.restype = _int

SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, q_weight: torch.Tensor, k_weight: torch.Tensor | None,
                 eps: float, table: torch.Tensor, positions: torch.Tensor, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """(q_out, k_out): each head of q and k normalised, weighted and turned by its token's position.

    The first table.shape[1] values of a head are turned, in pairs (i, i + rot/2), or
    (2i, 2i + 1) with interleaved=True.  Outputs have the inputs' dtype; pass q_out=q,
    k_out=k to work in place.  A negative position marks a padding token (zeros out).
    """
    if stream is None:
        return native.qk_norm_rope(q, k, q_weight, k_weight, eps, table, positions, interleaved, q_out, k_out)
    return on_stream(stream, native.qk_norm_rope, q, k, q_weight, k_weight, eps, table, positions, interleaved, q_out, k_out)


def rope(q: torch.Tensor, k: torch.Tensor | None, table: torch.Tensor, positions: torch.Tensor,
         interleaved: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """(q_out, k_out): qk_norm_rope's rotation alone."""
    if stream is None:
        return native.rope(q, k, table, positions, interleaved, False, q_out, k_out)
    return on_stream(stream, native.rope, q, k, table, positions, interleaved, False, q_out, k_out)


def rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor | None, table: torch.Tensor, positions: torch.Tensor,
                  interleaved: bool = False, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                  stream=None):
    """(dq, dk): rope's gradients, the transposed rotation of the outputs' gradients."""
    if stream is None:
        return native.rope(dq_out, dk_out, table, positions, interleaved, True, dq, dk)
    return on_stream(stream, native.rope, dq_out, dk_out, table, positions, interleaved, True, dq, dk)


def qk_backward_workspace_bytes(head_dim: int) -> int:
    n = lib.far_qk_backward_workspace_bytes(head_dim)
    if n < 0:
        raise FarError(-n)
    return n


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor | None, q: torch.Tensor, k: torch.Tensor | None,
                          q_weight: torch.Tensor, k_weight: torch.Tensor | None, eps: float, table: torch.Tensor,
                          positions: torch.Tensor, interleaved: bool = False, dq: torch.Tensor | None = None,
                          dk: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """(dq, dk, dq_weight, dk_weight): the gradients of qk_norm_rope given those of its outputs.

    q and k are the forward call's inputs.  The weights' gradients are float32, summed over
    tokens and heads in a fixed order.  workspace: qk_backward_workspace_bytes(head_dim)
    bytes, allocated when not given; calls that may overlap need one each.
    """
    args = (dq_out, dk_out, q, k, q_weight, k_weight, eps, table, positions, interleaved, dq, dk, workspace)
    return native.qk_norm_rope_backward(*args) if stream is None else on_stream(stream, native.qk_norm_rope_backward, *args)


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: dict | None = None) -> tuple[list, float]:
    """(frequencies, attention factor) of far_rope_frequencies.

    scaling: None, or {"type": "linear" | "ntk", "factor": a}, {"type": "yarn", "factor": a,
    "trained": length, "fast": 32, "slow": 1, "attention_factor": 0 for 0.1 ln(a) + 1}, or
    {"type": "bands", "factor": a, "trained": length, "low": 1, "high": 4}.
    """
    kind = "plain" if scaling is None else scaling["type"]
    if kind not in SCALINGS:
        raise ValueError(f"unknown scaling {kind!r}: one of {', '.join(SCALINGS)}")
    given = {} if scaling is None else {k: v for k, v in scaling.items() if k != "type"}
    want = {"plain": {}, "linear": {"factor": None}, "ntk": {"factor": None},
            "yarn": {"factor": None, "trained": None, "fast": 32.0, "slow": 1.0, "attention_factor": 0.0},
            "bands": {"factor": None, "trained": None, "low": 1.0, "high": 4.0}}[kind]
    for name in given:
        if name not in want:
            raise ValueError(f"scaling {kind!r} has no {name!r}")
    values = [given.get(name, default) for name, default in want.items()]
    if None in values:
        raise ValueError(f"scaling {kind!r} needs {', '.join(n for n, v in want.items() if v is None)}")
    params = (ctypes.c_double * max(1, len(values)))(*values)
    freq = (ctypes.c_double * max(1, rot_dim // 2))()
    factor = ctypes.c_double(0.0)
    _check(lib.far_rope_frequencies(rot_dim, base, SCALINGS[kind], ctypes.addressof(params), ctypes.addressof(freq),
                                    ctypes.addressof(factor)))
    return list(freq), factor.value


def rope_table(rows: int, rot_dim: int, base: float = 10000.0, scaling: dict | None = None, first_position: int = 0,
               device="cuda", stream=None) -> torch.Tensor:
    """The float32 [rows, rot_dim] table (cosines, then sines) for positions first_position ..,
    each value rounded once from binary64; made once, kept by the program."""
    freq, factor = rope_frequencies(rot_dim, base, scaling)
    if rows < 0:
        raise FarError(4)
    host = (ctypes.c_double * len(freq))(*freq)
    if torch.device(device).type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if stream is not None and torch.device(device).index not in (None, stream.device.index):
        raise ValueError("the stream belongs to another device than the tensors")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        here = torch.cuda.current_stream()
        table = torch.empty((rows, rot_dim), dtype=torch.float32, device=here.device)
        _check(lib.rope_table(table.data_ptr(), rows, rot_dim, first_position, ctypes.addressof(host), factor,
                              here.cuda_stream))
    if stream is not None:
        table.record_stream(torch.cuda.current_stream(table.device))
    return table
