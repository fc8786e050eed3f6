"""Recurrent states kept in 8 bits, slot by slot (include/gdn2.h,
gdn2_state_cache_*): stored after a prefill, loaded as the S0 or h0 of the
call that resumes from them.

A row (the last axis) shares one power-of-two scale; `fmt` is "e4m3" or "int8".
"""
from __future__ import annotations

import ctypes
import math

from . import GDN2_OK, Gdn2Error, _ptr, load
from ._launch import launch_on, want
from .linear import _ref

CACHE_FORMATS = {"e4m3": 0, "int8": 1}


class gdn2_cache_desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("P", ctypes.c_int32), ("rows", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("format", ctypes.c_int32)]


def declare(lib):
    vp, dp = ctypes.c_void_p, ctypes.POINTER(gdn2_cache_desc)
    for nm in ("store", "load"):
        f = getattr(lib, f"gdn2_state_cache_{nm}")
        f.restype, f.argtypes = ctypes.c_int, [dp] + [vp] * 4 + [vp]


# ------------------------------------------------------------------ raw C ABI
def gdn2_state_cache_store(desc, S, slots, cache, scales, stream=0) -> int:
    return load().gdn2_state_cache_store(_ref(desc), S, slots, cache, scales, stream)


def gdn2_state_cache_load(desc, cache, scales, slots, S, stream=0) -> int:
    return load().gdn2_state_cache_load(_ref(desc), cache, scales, slots, S, stream)


# ------------------------------------------------------------------ torch conveniences
def state_cache_empty(P, *shape, device=None):
    """(cache, scales) of P empty slots for states of `shape` (e.g. H_v, d_k,
    d_v): uint8 [P, *shape] and [P, *shape[:-1]], cleared (every slot reads
    back as zeros)."""
    import torch
    dev = torch.device("cuda") if device is None else device
    return (torch.zeros((P,) + shape, dtype=torch.uint8, device=dev),
            torch.zeros((P,) + shape[:-1], dtype=torch.uint8, device=dev))


def _problem(cache, scales, slots, fmt):
    import torch
    if fmt not in CACHE_FORMATS:
        raise ValueError(f"unknown cache format {fmt}")
    if cache.dim() < 3:
        raise ValueError(f"cache must be [P, ..., rows, d_v], got {tuple(cache.shape)}")
    dev = cache.device
    want(cache, "cache", cache.shape, torch.uint8, dev)
    want(scales, "scales", cache.shape[:-1], torch.uint8, dev)
    want(slots, "slots", (slots.numel(),), torch.int32, dev)
    return gdn2_cache_desc(slots.numel(), cache.shape[0], math.prod(cache.shape[1:-1]), cache.shape[-1],
                           CACHE_FORMATS[fmt]), dev


def state_cache_store(S, slots, cache, scales, fmt: str = "e4m3", stream=None):
    """S [N, ..., rows, d_v] fp32 into slots [N] (int32) of cache ([P, ...] like S,
    uint8) and scales ([P, ..., rows] uint8). Slots outside [0, P) are skipped;
    of entries with the same slot the last is kept."""
    import torch
    desc, dev = _problem(cache, scales, slots, fmt)
    want(S, "S", (desc.N,) + tuple(cache.shape[1:]), torch.float32, dev)
    with launch_on(dev, stream) as handle:
        st = gdn2_state_cache_store(desc, _ptr(S), _ptr(slots), _ptr(cache), _ptr(scales), handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)


def state_cache_load(cache, scales, slots, S=None, fmt: str = "e4m3", stream=None):
    """The states of `slots`, fp32 [N, ..., rows, d_v]; zeros for a slot outside [0, P)."""
    import torch
    desc, dev = _problem(cache, scales, slots, fmt)
    shape = (desc.N,) + tuple(cache.shape[1:])
    with launch_on(dev, stream) as handle:
        if S is None:
            S = torch.empty(shape, dtype=torch.float32, device=dev)
        else:
            want(S, "S", shape, torch.float32, dev)
        st = gdn2_state_cache_load(desc, _ptr(cache), _ptr(scales), _ptr(slots), _ptr(S), handle)
    if st != GDN2_OK:
        raise Gdn2Error(st)
    return S
