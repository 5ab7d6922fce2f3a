"""A layer's buffers, one set per shape of its input, in bounded memory."""

from __future__ import annotations

from collections import OrderedDict
from typing import Callable

import torch

KEEP_BYTES = 8 << 30  # of the sets that are kept; a step of 8192 tokens, 80 experts, top-8 takes 1.7 GB


def _tensors(o):
    if isinstance(o, torch.Tensor):
        yield o
    elif isinstance(o, dict):
        for v in o.values():
            yield from _tensors(v)
    elif isinstance(o, (tuple, list)):
        for v in o:
            yield from _tensors(v)


def _capturing() -> bool:
    return torch.cuda.is_current_stream_capturing()


def _current_stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index if device.index is not None else torch._C._cuda_getDevice())


class Buffers(OrderedDict):
    """Buffer sets by key, least recently used first; sets beyond ``keep_bytes`` in all are dropped, oldest first.

    The set in use stays whatever its size, and so does one that a HIP graph was captured with: the graph holds its
    addresses.  A dropped set's memory goes back to the pool of the stream it was made on; where another stream has
    used it, the allocator is told, and hands it on only after that stream's work.  Tensors that a caller still holds
    are not affected: they keep their memory."""

    def __init__(self, device, keep_bytes: int = KEEP_BYTES):
        super().__init__()
        self.device, self.keep_bytes = torch.device(device), keep_bytes
        self.bytes = 0  # of the sets that may be dropped
        self._size: dict = {}  # key -> bytes, without the captured sets
        self._stream: dict = {}  # key -> the stream it was made on

    def take(self, key, make: Callable[[], dict]) -> dict:
        """The set of `key`, made by make() if there is none, for use on the current stream."""
        b = self.get(key)
        if b is None:
            b = self[key] = make()
            self._size[key] = sum(t.numel() * t.element_size() for t in _tensors(b))
            self._stream[key] = _current_stream(self.device)
            self.bytes += self._size[key]
        else:
            self.move_to_end(key)
        if _capturing():
            self.bytes -= self._size.pop(key, 0)
        elif key in self._size and self._stream[key] != _current_stream(self.device):
            for t in _tensors(b):
                t.record_stream(torch.cuda.current_stream(self.device))
        if self.bytes > self.keep_bytes:
            self._drop(key)
        return b

    def _drop(self, used) -> None:
        for key in [k for k in self if k in self._size and k != used]:
            if self.bytes <= self.keep_bytes:
                return
            self.bytes -= self._size.pop(key)
            del self._stream[key], self[key]
