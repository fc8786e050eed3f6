"""Where a call of the torch conveniences runs: the tensors' device and a stream of it."""
from __future__ import annotations


class launch_on:
    """with launch_on(device, stream) as handle: the tensors' device is current,
    new tensors belong to the launch's stream, and handle is that stream's
    address. `stream`: a torch stream, a raw hipStream_t, or None (the device's
    current stream)."""

    __slots__ = ("_dev", "_stream", "_ctx")

    def __init__(self, device, stream):
        self._dev, self._stream, self._ctx = device, stream, ()

    def __enter__(self):
        import torch
        if self._stream is None:
            if torch.cuda.current_device() != self._dev.index:
                ctx = torch.cuda.device(self._dev)
                ctx.__enter__()
                self._ctx = (ctx,)
            return torch.cuda.current_stream(self._dev).cuda_stream
        s = self._stream
        if not hasattr(s, "cuda_stream"):
            s = (torch.cuda.ExternalStream(int(s), device=self._dev) if int(s)
                 else torch.cuda.default_stream(self._dev))
        if s.device.index != self._dev.index:
            raise ValueError(f"stream is of {s.device}, but the tensors are on {self._dev}")
        ctx = torch.cuda.stream(s)  # makes its device current as well
        ctx.__enter__()
        self._ctx = (ctx,)
        return s.cuda_stream

    def __exit__(self, *exc):
        for ctx in self._ctx:
            ctx.__exit__(*exc)
        return False
