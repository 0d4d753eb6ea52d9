"""Thin ctypes binding of the row calls in libsrm_moe.so (declared in
include/srm_rows.h): token rows sorted by expert and back with the routing
weights applied, and the gradients of both.

Argument marshalling only: every step runs in the library's CUDA kernels;
PyTorch supplies device memory and the current stream of the tensors' device.
No fallback: if the library is missing, every call raises.

    cfg = rows.Config(T, H, E, K)                     # tokens bf16, experts' rows fp16
    counts, offsets, sorted_ = moe.permute(block_cfg, idx, ws)
    xs, pos = rows.sort(cfg, x, offsets, sorted_, ws)
    ys = ...                                          # each group's product of its rows of xs
    y = rows.unsort(cfg, ys, gate, pos, ws, residual=x)
    dys, dgate = rows.unsort_grad(cfg, dy, ys, gate, pos, ws)
    dx = rows.sort_grad(cfg, dxs, pos, ws)            # dxs: from dys through the products

``ws`` is a workspace of this library (its error word takes what only the
device can see; read it with moe.device_error) or rows.workspace().
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import moe
from .q8 import DTYPES, FLOATS, _ld, _on, _rows, _vector

SYMBOLS = ("moe_rows_sort", "moe_rows_unsort", "moe_rows_sort_grad", "moe_rows_unsort_grad")


class _Cfg(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("E", ctypes.c_int32), ("K", ctypes.c_int32),
                ("has_shared", ctypes.c_int32), ("dtype", ctypes.c_int32), ("slot_dtype", ctypes.c_int32),
                ("ld_token", ctypes.c_int64), ("ld_slot", ctypes.c_int64), ("ld_residual", ctypes.c_int64),
                ("ld_dys", ctypes.c_int64)]


@dataclasses.dataclass(frozen=True)
class Config:
    """T tokens, rows of H elements, E experts, K per token; dtype of the tokens' rows (sort also takes
    int8), slot_dtype of the experts' rows that unsort reads."""
    T: int
    H: int
    E: int
    K: int
    has_shared: bool = True
    dtype: torch.dtype = torch.bfloat16
    slot_dtype: torch.dtype = torch.float16

    @classmethod
    def of(cls, cfg: moe.Config, **kw) -> "Config":
        """The row calls of a block configuration."""
        return cls(cfg.T, cfg.H, cfg.E, cfg.K, cfg.has_shared, **kw)

    @property
    def rows(self) -> int:
        """Expert-sorted positions: T*K routed plus T shared."""
        return self.T * self.K + (self.T if self.has_shared else 0)

    def c(self, token, slot, residual=None, dys=None) -> _Cfg:
        return _Cfg(self.T, self.H, self.E, self.K, int(bool(self.has_shared)), DTYPES.get(self.dtype, -1),
                    DTYPES.get(self.slot_dtype, -1), _ld(token), _ld(slot), _ld(residual), _ld(dys))


_bound = False


def lib():
    """The library with the row entry points typed."""
    global _bound
    L = moe.lib()
    if not _bound:
        vp, P = ctypes.c_void_p, ctypes.POINTER
        for name, n in (("moe_rows_sort", 9), ("moe_rows_unsort", 7), ("moe_rows_sort_grad", 5),
                        ("moe_rows_unsort_grad", 8)):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [P(_Cfg)] + [vp] * n
        _bound = True
    return L


def workspace(device=None) -> torch.Tensor:
    """A zeroed control block for calls without another workspace (256 bytes)."""
    return torch.zeros(256, dtype=torch.uint8, device=device or "cuda")


def _ws(ws, device):
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.numel() < 256:
        raise TypeError("ws must be a uint8 tensor of at least 256 bytes")
    if ws.device != device:
        raise ValueError("ws is on %s, the call on %s" % (ws.device, device))
    return moe._ptr(ws)


def _out(out, name, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _rows(out, name, shape, (dtype,), device)


def sort(cfg: Config, x, offsets, sorted_, ws, x_scale=None, out=None, pos=None, xs_scale=None, stream=None):
    """Token rows x [T, H] in expert-sorted order: (xs [rows, H], pos int32 [rows]), or with the scales of
    8-bit rows (x_scale fp32 [T]) (xs, xs_scale fp32 [rows], pos).  pos is the inverse of sorted_."""
    _rows(x, "x", (cfg.T, cfg.H), (cfg.dtype,))
    dev = x.device
    _vector(offsets, "offsets", cfg.E + 2, torch.int32, dev)
    _vector(sorted_, "sorted", cfg.rows, torch.int32, dev)
    if x_scale is not None:
        _vector(x_scale, "x_scale", cfg.T, torch.float32, dev)
    with _on(dev, stream):
        xs = _out(out, "out", (cfg.rows, cfg.H), cfg.dtype, dev)
        if pos is None:
            pos = torch.empty((cfg.rows,), dtype=torch.int32, device=dev)
        _vector(pos, "pos", cfg.rows, torch.int32, dev)
        if x_scale is not None:
            if xs_scale is None:
                xs_scale = torch.empty((cfg.rows,), dtype=torch.float32, device=dev)
            _vector(xs_scale, "xs_scale", cfg.rows, torch.float32, dev)
        elif xs_scale is not None:
            raise ValueError("xs_scale without x_scale")
        moe._check(lib().moe_rows_sort(ctypes.byref(cfg.c(x, xs)), moe._ptr(x), moe._ptr(x_scale),
                                       moe._ptr(offsets), moe._ptr(sorted_), moe._ptr(pos), moe._ptr(xs),
                                       moe._ptr(xs_scale), _ws(ws, dev), moe._stream(stream)), "moe_rows_sort")
    return (xs, pos) if x_scale is None else (xs, xs_scale, pos)


def unsort(cfg: Config, ys, gate, pos, ws, residual=None, out=None, stream=None):
    """y [T, H] = (residual +) sum over slots of gate * ys[pos] + the shared row; gate fp32 [T, K], or None
    for weights 1.  ``out`` may be the residual itself."""
    _rows(ys, "ys", (cfg.rows, cfg.H), (cfg.slot_dtype,))
    dev = ys.device
    _pos_gate(cfg, pos, gate, dev)
    if residual is not None:
        _rows(residual, "residual", (cfg.T, cfg.H), (cfg.dtype,), dev)
    with _on(dev, stream):
        y = _out(out, "out", (cfg.T, cfg.H), cfg.dtype, dev)
        moe._check(lib().moe_rows_unsort(ctypes.byref(cfg.c(y, ys, residual)), moe._ptr(ys), moe._ptr(gate),
                                         moe._ptr(pos), moe._ptr(residual), moe._ptr(y), _ws(ws, dev),
                                         moe._stream(stream)), "moe_rows_unsort")
    return y


def sort_grad(cfg: Config, dxs, pos, ws, out=None, stream=None):
    """dx [T, H] from the sorted rows' gradients dxs [rows, H] (both of cfg.dtype)."""
    _rows(dxs, "dxs", (cfg.rows, cfg.H), (cfg.dtype,))
    dev = dxs.device
    _pos_gate(cfg, pos, None, dev)
    with _on(dev, stream):
        dx = _out(out, "out", (cfg.T, cfg.H), cfg.dtype, dev)
        moe._check(lib().moe_rows_sort_grad(ctypes.byref(cfg.c(dx, dxs)), moe._ptr(dxs), moe._ptr(pos),
                                            moe._ptr(dx), _ws(ws, dev), moe._stream(stream)),
                   "moe_rows_sort_grad")
    return dx


def unsort_grad(cfg: Config, dy, ys, gate, pos, ws, out=None, dgate=None, stream=None):
    """(dys [rows, H] of slot_dtype, dgate fp32 [T, K]) from dy [T, H].  ``out`` may be ys itself; rows
    that no assignment holds are left as they were."""
    _rows(dy, "dy", (cfg.T, cfg.H), (cfg.dtype,))
    dev = dy.device
    _rows(ys, "ys", (cfg.rows, cfg.H), (cfg.slot_dtype,), dev)
    _pos_gate(cfg, pos, gate, dev)
    with _on(dev, stream):
        dys = _out(out, "out", (cfg.rows, cfg.H), cfg.slot_dtype, dev)
        if dgate is None:
            dgate = torch.empty((cfg.T, cfg.K), dtype=torch.float32, device=dev)
        moe._req(dgate, torch.float32, (cfg.T, cfg.K), "dgate")
        moe._check(lib().moe_rows_unsort_grad(ctypes.byref(cfg.c(dy, ys, dys=dys)), moe._ptr(dy), moe._ptr(ys),
                                              moe._ptr(gate), moe._ptr(pos), moe._ptr(dys), moe._ptr(dgate),
                                              _ws(ws, dev), moe._stream(stream)), "moe_rows_unsort_grad")
    return dys, dgate


def _pos_gate(cfg, pos, gate, device):
    _vector(pos, "pos", cfg.rows, torch.int32, device)
    if gate is not None:
        moe._req(gate, torch.float32, (cfg.T, cfg.K), "gate")
        if gate.device != device:
            raise ValueError("gate is on %s, the call on %s" % (gate.device, device))
