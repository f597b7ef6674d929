"""The native binding of the per-head and block-scaled operators, and their explicit streams.

``_build/_far_torch.so`` (csrc/far_torch.cpp) checks a call's tensors, allocates its outputs and
enqueues it on the tensors' device, whatever the current one is, and that device's current
stream.  It is loaded by the first call that needs it: the other operators go through ctypes
and ``libfar.so`` alone, and stay usable where this module is missing or was built for
another PyTorch (such a call then fails, and says so).

A call with ``stream=`` runs with that stream current: outputs are allocated on it,
and the inputs (and the outputs, for the stream that was current) are recorded, so that the
caching allocator hands none of that memory out again before both streams are done with it;
ordering the two streams is the caller's part, as for any work on two streams.
"""
from __future__ import annotations

import importlib.util
import os
import threading

import torch

from . import FarError, _PKG

BINDING_PATH = os.path.join(_PKG, "_build", "_far_torch.so")
_loading = threading.Lock()


def _load():
    rebuild = "build it for this PyTorch (python -c 'import __graft_entry__ as g; g.build()')"
    if not os.path.exists(BINDING_PATH):
        raise ImportError(f"{BINDING_PATH} is missing: {rebuild}")
    spec = importlib.util.spec_from_file_location("_far_torch", BINDING_PATH)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        raise ImportError(f"{BINDING_PATH} cannot be loaded ({e}): {rebuild}") from e
    module.init_errors(FarError, torch.OutOfMemoryError)
    return module


class _Native:
    """The binding's functions, looked up when they are first called (later ones find them in the instance)."""

    def __getattr__(self, name):
        with _loading:
            module = self.__dict__.get("_module")
            if module is None:
                module = self._module = _load()
        function = getattr(module, name)
        setattr(self, name, function)
        return function


native = _Native()


def on_stream(stream, call, *args):
    """call(*args) on an explicit stream."""
    tensors = [a for a in args if isinstance(a, torch.Tensor)]
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        if t.device != stream.device:
            raise ValueError("the stream belongs to another device than the tensors")
    here = torch.cuda.current_stream(stream.device)
    if stream == here:
        return call(*args)
    with torch.cuda.stream(stream):
        out = call(*args)
    for t in tensors:
        t.record_stream(stream)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and not any(t is a for a in tensors):
            t.record_stream(here)
    return out
