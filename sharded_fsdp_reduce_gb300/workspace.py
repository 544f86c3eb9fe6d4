"""Device memory that an object's calls work in, on any stream."""
from __future__ import annotations

from typing import Optional

import torch

__all__ = ["Workspace", "take"]


def take(nbytes: int, device, alignment: int = 256, zeroed: bool = False) -> torch.Tensor:
    """nbytes of the allocator's memory at a multiple of `alignment`, in the
    current stream's order."""
    make = torch.zeros if zeroed else torch.empty
    if alignment <= 256:  # every CUDA allocation's
        return make(nbytes, dtype=torch.uint8, device=device)
    whole = make(nbytes + alignment, dtype=torch.uint8, device=device)
    return whole.narrow(0, -whole.data_ptr() % alignment, nbytes)


class Workspace:
    """nbytes of device memory at a multiple of `alignment`, that calls on any
    stream may use, in order; zeroed, or with whatever it holds. The memory may
    have had another user on the stream it is taken on, whose work is still
    queued there: other streams wait for that."""

    def __init__(self, nbytes: int, device, alignment: int = 256, zeroed: bool = False):
        self.buf = take(nbytes, device, alignment, zeroed)
        self._device = self.buf.get_device()
        self._zeroed = zeroed
        self._in_capture = torch.cuda.is_current_stream_capturing()
        self._mark(torch.cuda.current_stream(self.buf.device))

    def _mark(self, stream: torch.cuda.Stream) -> None:
        self._made_on = stream.cuda_stream
        self._ready = stream.record_event()

    def check_device(self) -> None:
        """The kernels run on the current device, which has to be the memory's."""
        if torch.cuda.current_device() != self._device:
            raise ValueError(f"this object's workspace is on cuda:{self._device} but the current device is "
                             f"cuda:{torch.cuda.current_device()}")

    def on(self, stream: Optional[torch.cuda.Stream]) -> torch.cuda.Stream:
        """The stream of a call (the current one by default), ordered after
        what the memory was used for before and holding it until its work is
        done."""
        self.check_device()
        s = stream if stream is not None else torch.cuda.current_stream()
        if self._in_capture and not torch.cuda.is_current_stream_capturing():
            # made within a capture: its zeroing and its event are the graph's,
            # which may not have run yet
            if self._zeroed:
                with torch.cuda.stream(s):
                    self.buf.zero_()
            self._in_capture = False
            self._mark(s)
        if s.cuda_stream != self._made_on:
            # (a capture starts after the device is idle and cannot wait for work outside it)
            if not torch.cuda.is_current_stream_capturing():
                s.wait_event(self._ready)
            self.buf.record_stream(s)
        return s
