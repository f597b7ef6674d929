"""Per-head RMSNorm of queries and keys with the rotation by position, its gradients, the
rotation alone, and the table of cosines and sines they read (ctypes binding; the contract
stands in ``include/far.h`` at qk_norm_rope).

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
import math

import torch

from . import TORCH_TO_CODE, FarError, _check, dtypes, lib
from ._launch import Launch, ptr

_vp, _f32, _i64, _int, _f64 = ctypes.c_void_p, ctypes.c_float, ctypes.c_int64, ctypes.c_int, ctypes.c_double
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

_NONE = (None, 0, 0)
SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


def _heads(t: torch.Tensor):
    """(pointer, token stride, head stride) of a [..., heads, dim] tensor."""
    if t.dim() == 3:
        n, h, d = t.shape
        ts, hs, ds = t.stride()
    else:
        if t.dim() < 3:
            raise ValueError("q and k are [..., heads, head_dim]")
        *lead, h, d = t.shape
        *ls, hs, ds = t.stride()
        n, ts = math.prod(lead), 0
        run = None  # the stride the axes inside would need to continue
        for size, st in zip(reversed(lead), reversed(ls)):
            if size == 1:
                continue
            if run is None:
                ts = st
            elif st != run and n > 0:
                raise ValueError("the leading axes do not collapse to one stride: call once a sequence, or copy")
            run = st * size
    if ds != 1 and d > 1:
        raise ValueError("the values of a head must be contiguous")
    return t.data_ptr(), (ts if n > 1 else 0), (hs if h > 1 else 0)


def _place(table, positions, tokens, rot):
    if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous():
        raise ValueError("table must be a contiguous float32 [rows, rot_dim] tensor (rope_table)")
    if positions.dtype not in (torch.int64, torch.int32) or not positions.is_contiguous():
        raise ValueError("positions must be a contiguous int32 or int64 tensor")
    if positions.numel() != tokens:
        raise ValueError("one position for each token")
    return table.data_ptr(), table.shape[0], positions.data_ptr(), positions.element_size()


def _sizes(q, k):
    """tokens, query heads, key heads, head_dim; the tensors' agreement."""
    if q.dim() < 3:
        raise ValueError("q and k are [..., heads, head_dim]")
    *lead, h, d = q.shape
    hk = 0
    if k is not None:
        if k.shape[:-2] != q.shape[:-2] or k.shape[-1] != d:
            raise ValueError("q and k must agree but in their number of heads")
        if k.dtype != q.dtype:
            raise ValueError("q and k must share a dtype")
        hk = k.shape[-2]
    n = lead[0] if len(lead) == 1 else math.prod(lead)
    return n, h, hk, d


def _outputs(go, q, k, q_out, k_out):
    """The outputs given, checked, or new ones."""
    outs = []
    for x, y in ((q, q_out), (k, k_out)):
        if x is None:
            if y is not None:
                raise ValueError("an output without its input")
        elif y is None:
            y = go.empty(x.shape, x.dtype)
        elif y.shape != x.shape or y.dtype != x.dtype:
            raise ValueError("an output has its input's shape and dtype")
        outs.append(y)
    return outs


def _pair_weights(q, k, q_weight, k_weight, d):
    for x, w in ((q, q_weight), (k, k_weight)):
        if x is not None and (w is None or w.numel() != d or not w.is_contiguous()):
            raise ValueError("a weight is a contiguous [head_dim] tensor")
    if k is not None and q_weight.dtype != k_weight.dtype:
        raise ValueError("q_weight and k_weight must share a dtype")
    return dtypes(q.dtype, q_weight.dtype)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, q_weight: torch.Tensor, k_weight: torch.Tensor | None,
                 eps: float, table: torch.Tensor, positions: torch.Tensor, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """(q_out, k_out): each head of q and k normalised, weighted and turned by its token's position.

    The first table.shape[1] values of a head are turned, in pairs (i, i + rot/2), or
    (2i, 2i + 1) with interleaved=True.  Outputs have the inputs' dtype; pass q_out=q,
    k_out=k to work in place.  A negative position marks a padding token (zeros out).
    """
    n, h, hk, d = _sizes(q, k)
    code = _pair_weights(q, k, q_weight, k_weight, d)
    go = Launch(stream, q, k, q_weight, k_weight, table, positions, q_out, k_out)
    yq, yk = _outputs(go, q, k, q_out, k_out)
    go.run(lib.qk_norm_rope, *_heads(q), *(_NONE if k is None else _heads(k)), ptr(q_weight), ptr(k_weight), eps,
           *_place(table, positions, n, d), *_heads(yq), *(_NONE if k is None else _heads(yk)), n, h, hk, d,
           table.shape[1], int(interleaved), code)
    return yq, yk


def _rope(q, k, table, positions, interleaved, transpose, q_out, k_out, stream):
    n, h, hk, d = _sizes(q, k)
    if q.dtype not in TORCH_TO_CODE:
        raise FarError(2)
    go = Launch(stream, q, k, table, positions, q_out, k_out)
    yq, yk = _outputs(go, q, k, q_out, k_out)
    go.run(lib.rope, *_heads(q), *(_NONE if k is None else _heads(k)), *_place(table, positions, n, d), *_heads(yq),
           *(_NONE if k is None else _heads(yk)), n, h, hk, d, table.shape[1], int(interleaved), transpose,
           TORCH_TO_CODE[q.dtype])
    return yq, yk


def rope(q: torch.Tensor, k: torch.Tensor | None, table: torch.Tensor, positions: torch.Tensor,
         interleaved: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """(q_out, k_out): qk_norm_rope's rotation alone."""
    return _rope(q, k, table, positions, interleaved, 0, q_out, k_out, stream)


def rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor | None, table: torch.Tensor, positions: torch.Tensor,
                  interleaved: bool = False, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                  stream=None):
    """(dq, dk): rope's gradients, the transposed rotation of the outputs' gradients."""
    return _rope(dq_out, dk_out, table, positions, interleaved, 1, dq, dk, stream)


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
    n, h, hk, d = _sizes(q, k)
    code = _pair_weights(q, k, q_weight, k_weight, d)
    for x, g in ((q, dq_out), (k, dk_out)):
        if (x is None) != (g is None) or (x is not None and (g.shape != x.shape or g.dtype != x.dtype)):
            raise ValueError("an output's gradient has its input's shape and dtype")
    go = Launch(stream, q, k, q_weight, k_weight, table, positions, dq_out, dk_out, dq, dk, workspace)
    yq, yk = _outputs(go, q, k, dq, dk)
    dw = go.empty((2 if k is not None else 1, d), torch.float32)
    if workspace is None:
        workspace = go.empty(qk_backward_workspace_bytes(d), torch.uint8)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    dqw = dw[0]
    dkw = dw[1] if k is not None else None
    none = _NONE if k is None else None
    go.run(lib.qk_norm_rope_backward, *_heads(dq_out), *(none or _heads(dk_out)), *_heads(q), *(none or _heads(k)),
           ptr(q_weight), ptr(k_weight), eps, *_place(table, positions, n, d), *_heads(yq), *(none or _heads(yk)),
           ptr(dqw), ptr(dkw), ptr(workspace), workspace.numel() * workspace.element_size(), n, h, hk, d,
           table.shape[1], int(interleaved), code)
    return yq, yk, dqw, dkw


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
    anchor = torch.empty(0, device=device)
    go = Launch(stream, anchor)
    table = go.empty((rows, rot_dim), torch.float32)
    go.run(lib.rope_table, ptr(table), rows, rot_dim, first_position, ctypes.addressof(host), factor)
    return table
