"""Where a call of the torch conveniences runs (the tensors' device and a stream
of it), and their argument check, kept short: for the smallest calls the host's
time is the call's time."""
from __future__ import annotations

from . import _want


def want(t, name, shape, dtype, device):
    """_want, with the tensors that pass told apart first."""
    if t is None:
        return
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
            return
    except AttributeError:
        pass
    _want(t, name, tuple(shape), dtype, device)


def no_second_order(name):
    """The gradients come from a kernel that autograd cannot see into; grad mode
    is on in a backward only for create_graph=True."""
    import torch
    if torch.is_grad_enabled():
        raise RuntimeError(f"{name} has no second derivatives (create_graph=True)")


class launch_on:
    """with launch_on(device, stream) as handle: the tensors' device is current,
    new tensors belong to the launch's stream, and handle is that stream's
    address. `stream`: a torch stream, a raw hipStream_t, or None (the device's
    current stream)."""

    __slots__ = ("_dev", "_stream", "_ctx")

    def __init__(self, device, stream):
        self._dev, self._stream, self._ctx = device, stream, None

    def __enter__(self):
        import torch
        s = self._stream
        if s is None:
            index = self._dev.index
            if torch._C._cuda_getDevice() != index:
                self._ctx = torch.cuda.device(self._dev)
                self._ctx.__enter__()
            return torch._C._cuda_getCurrentRawStream(index)
        if not hasattr(s, "cuda_stream"):
            s = (torch.cuda.ExternalStream(int(s), device=self._dev) if int(s)
                 else torch.cuda.default_stream(self._dev))
        if s.device.index != self._dev.index:
            raise ValueError(f"stream is of {s.device}, but the tensors are on {self._dev}")
        self._ctx = torch.cuda.stream(s)  # makes its device current as well
        self._ctx.__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        return False
