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


def layout_of(*tensors):
    """Strides of saved tensors: what hooks on them may return otherwise than it
    was (the same values, sizes and type, laid out as the hook's copy has them)."""
    return [None if t is None else t.stride() for t in tensors]


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


def want_tokens(t, name, shape, dtype, device):
    """t must be `shape` [..., heads, d] on `device` with every token's heads
    contiguous and the tokens one distance apart; that distance in elements."""
    try:  # the tensors that pass, told apart first
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index:
            st, (H, d) = t.stride(), shape[-2:]
            if st[-1] == 1 and st[-2] == d and (len(st) == 3 or (len(st) == 4 and (st[0] == shape[1] * st[1]))):
                if st[-3] >= H * d:
                    return st[-3]
    except AttributeError:
        pass
    import torch
    if t.is_contiguous():
        want(t, name, shape, dtype, device)
        return t.shape[-2] * t.shape[-1]
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a torch tensor on a GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, but q is on {device}")
    *lead, H, d = t.shape
    *steps, head, one = t.stride()
    if t.numel() == 0:
        return H * d
    step = reach = None
    for n, s in zip(reversed(lead), reversed(steps)):
        if n == 1:
            continue
        if step is None:
            step, reach = s, s * n
        elif s != reach:
            step = -1
            break
        else:
            reach *= n
    if step is None:
        step = H * d
    if (d > 1 and one != 1) or (H > 1 and head != d) or step < H * d:
        raise ValueError(f"{name} must hold each token's [heads, d] contiguously and its tokens one distance apart, "
                         f"got strides {t.stride()} for shape {tuple(t.shape)}")
    return step
