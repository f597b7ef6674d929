"""What the bindings of the per-head and block-scaled operators share: device and stream of a call.

A call runs on its tensors' device, whatever the current one is, and on `stream` or that
device's current stream.  With an explicit stream that is not the current one, outputs are
allocated on it, and the inputs (and the outputs, for the current stream) are recorded, so
that the caching allocator hands none of that memory out again before both streams are done
with it; ordering the two streams is the caller's part, as for any work on two streams.
"""
from __future__ import annotations

import torch

from . import _check

_raw_stream = torch._C._cuda_getCurrentRawStream


def device_of(*tensors) -> int:
    """The one CUDA device all tensors (None: not given) are on."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d < 0:
                raise ValueError("tensors must be on a CUDA device")
            if dev is None:
                dev = d
            elif d != dev:
                raise ValueError("tensors must be on one device")
    return dev


class Launch:
    """The device and stream of one call; `inputs` are what it reads."""

    __slots__ = ("dev", "handle", "stream", "other")

    def __init__(self, stream, *tensors):
        self.dev = dev = device_of(*tensors)
        current = _raw_stream(dev)
        self.stream = stream
        if stream is None:
            self.handle, self.other = current, False
            return
        if stream.device.index != dev:
            raise ValueError("the stream belongs to another device than the tensors")
        self.handle = stream.cuda_stream
        self.other = self.handle != current
        if self.other:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def empty(self, shape, dtype):
        """An output or workspace of this call."""
        if not self.other:
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.dev))
        here = torch.cuda.current_stream(self.dev)
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.dev))
        t.record_stream(here)
        return t

    def run(self, fn, *args) -> None:
        if self.dev == torch.cuda.current_device():
            _check(fn(*args, self.handle))
        else:
            with torch.cuda.device(self.dev):
                _check(fn(*args, self.handle))


def ptr(t):
    return None if t is None else t.data_ptr()
