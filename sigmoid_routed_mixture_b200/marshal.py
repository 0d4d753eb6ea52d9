"""Argument marshalling shared by the row and product bindings (q8, rows).

A decode step's kernels take a few microseconds, so the checks are written to
cost less than a launch: each returns the address (and row stride) it has just
checked, and looks closer only where the common case does not hold.
"""
from __future__ import annotations

import torch

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3}
FLOATS = (torch.bfloat16, torch.float16, torch.float32)


def elsewhere(t, stream) -> bool:
    """Whether a call on ``t`` needs another device or stream than the current one; ``t`` is checked to
    be a CUDA tensor.  The call then runs again inside ``on(t, stream)``, where it does not."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor, got %s" % type(t).__name__)
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device, got %s" % t.device)
    return stream is not None or t.get_device() != _current_device()


def on(t, stream):
    """The tensors' device and the call's stream as the current ones, so that what the call allocates
    belongs to them."""
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError("stream is on %s, the tensors are on %s" % (stream.device, t.device))
    return torch.cuda.stream(stream)


# the current stream of a device, as an address
raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice  # CUDA is up: there is a CUDA tensor


def mat(t, name, shape, dtype, device):
    """(address, row stride) of a matrix `shape` of `dtype` with contiguous rows on CUDA device `device`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr(), shape[1]
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % name) from None
    _check(t, name, shape, dtype, device)
    if shape[1] > 1 and t.stride(1) != 1 and shape[0] > 0:
        raise ValueError("%s must have contiguous rows" % name)
    if shape[0] > 1 and t.stride(0) < shape[1]:
        raise ValueError("%s must have rows that do not overlap" % name)
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]


def vec(t, name, shape, dtype, device) -> int:
    """The address of a contiguous tensor `shape` of `dtype` on CUDA device `device`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError("%s must be a torch.Tensor" % name) from None
    _check(t, name, shape, dtype, device)
    raise ValueError("%s must be contiguous" % name)


def _check(t, name, shape, dtype, device):
    if t.get_device() != device:
        raise ValueError("%s is on %s, the call on cuda:%d" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def rows_of(t, name, dtypes):
    """(T, H) of a matrix of one of the `dtypes`."""
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(map(str, dtypes)), t.dtype))
    if t.dim() != 2:
        raise ValueError("%s must have shape [T, H], got %s" % (name, tuple(t.shape)))
    return t.shape


def workspace(ws, least, device) -> int:
    """The address of a uint8 workspace of at least `least` bytes."""
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.numel() < least:
        raise TypeError("ws must be a uint8 tensor of at least %d bytes" % least)
    if ws.get_device() != device:
        raise ValueError("ws is on %s, the call on cuda:%d" % (ws.device, device))
    return ws.data_ptr()
