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
from .marshal import DTYPES, elsewhere, mat, on, raw_stream, vec
from .marshal import workspace as workspace_ptr

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

    def c(self, ld_token, ld_slot, ld_residual=0, ld_dys=0) -> _Cfg:
        return _Cfg(self.T, self.H, self.E, self.K, 1 if self.has_shared else 0, DTYPES.get(self.dtype, -1),
                    DTYPES.get(self.slot_dtype, -1), ld_token, ld_slot, ld_residual, ld_dys)


_lib = None


def lib():
    """The library with the row entry points typed."""
    global _lib
    if _lib is None:
        L = moe.lib()
        vp, P = ctypes.c_void_p, ctypes.POINTER
        for name, n in (("moe_rows_sort", 9), ("moe_rows_unsort", 7), ("moe_rows_sort_grad", 5),
                        ("moe_rows_unsort_grad", 8)):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [P(_Cfg)] + [vp] * n
        _lib = L
    return _lib


def workspace(device=None) -> torch.Tensor:
    """A zeroed control block for calls without another workspace (256 bytes)."""
    return torch.zeros(256, dtype=torch.uint8, device=device or "cuda")


def _pos_gate(cfg, pos, gate, dev):
    pos_ptr = vec(pos, "pos", (cfg.rows,), torch.int32, dev)
    return pos_ptr, vec(gate, "gate", (cfg.T, cfg.K), torch.float32, dev) if gate is not None else None


def _mat_out(out, like, name, shape, dtype, dev):
    if out is None:
        out = like.new_empty(shape, dtype=dtype)
        return out, out.data_ptr(), shape[1]
    return out, *mat(out, name, shape, dtype, dev)


def _vec_out(out, like, name, shape, dtype, dev):
    if out is None:
        out = like.new_empty(shape, dtype=dtype)
        return out, out.data_ptr()
    return out, vec(out, name, shape, dtype, dev)


def sort(cfg: Config, x, offsets, sorted_, ws, x_scale=None, out=None, pos=None, xs_scale=None, stream=None):
    """Token rows x [T, H] in expert-sorted order: (xs [rows, H], pos int32 [rows]), or with the scales of
    8-bit rows (x_scale fp32 [T]) (xs, xs_scale fp32 [rows], pos).  pos is the inverse of sorted_."""
    if elsewhere(x, stream):
        with on(x, stream):
            return sort(cfg, x, offsets, sorted_, ws, x_scale, out, pos, xs_scale)
    P, H, t, dev = cfg.rows, cfg.H, cfg.dtype, x.get_device()
    x_ptr, ld = mat(x, "x", (cfg.T, H), t, dev)
    off_ptr = vec(offsets, "offsets", (cfg.E + 2,), torch.int32, dev)
    ids_ptr = vec(sorted_, "sorted", (P,), torch.int32, dev)
    ws_ptr = workspace_ptr(ws, 256, dev)
    xs, xs_ptr, ld_s = _mat_out(out, x, "out", (P, H), t, dev)
    pos, pos_ptr = _vec_out(pos, x, "pos", (P,), torch.int32, dev)
    scale_ptr = xs_scale_ptr = None
    if x_scale is not None:
        scale_ptr = vec(x_scale, "x_scale", (cfg.T,), torch.float32, dev)
        xs_scale, xs_scale_ptr = _vec_out(xs_scale, x, "xs_scale", (P,), torch.float32, dev)
    elif xs_scale is not None:
        raise ValueError("xs_scale without x_scale")
    rc = (_lib or lib()).moe_rows_sort(cfg.c(ld, ld_s), x_ptr, scale_ptr, off_ptr, ids_ptr, pos_ptr, xs_ptr,
                                       xs_scale_ptr, ws_ptr, raw_stream(dev))
    if rc:
        raise moe.MoeError(rc, "moe_rows_sort")
    return (xs, pos) if x_scale is None else (xs, xs_scale, pos)


def unsort(cfg: Config, ys, gate, pos, ws, residual=None, out=None, stream=None):
    """y [T, H] = (residual +) sum over slots of gate * ys[pos] + the shared row; gate fp32 [T, K], or None
    for weights 1.  ``out`` may be the residual itself."""
    if elsewhere(ys, stream):
        with on(ys, stream):
            return unsort(cfg, ys, gate, pos, ws, residual, out)
    shape, t, dev = (cfg.T, cfg.H), cfg.dtype, ys.get_device()
    ys_ptr, ld_s = mat(ys, "ys", (cfg.rows, cfg.H), cfg.slot_dtype, dev)
    pos_ptr, gate_ptr = _pos_gate(cfg, pos, gate, dev)
    r_ptr, ld_r = mat(residual, "residual", shape, t, dev) if residual is not None else (None, 0)
    ws_ptr = workspace_ptr(ws, 256, dev)
    y, y_ptr, ld = _mat_out(out, ys, "out", shape, t, dev)
    rc = (_lib or lib()).moe_rows_unsort(cfg.c(ld, ld_s, ld_r), ys_ptr, gate_ptr, pos_ptr, r_ptr, y_ptr, ws_ptr,
                                         raw_stream(dev))
    if rc:
        raise moe.MoeError(rc, "moe_rows_unsort")
    return y


def sort_grad(cfg: Config, dxs, pos, ws, out=None, stream=None):
    """dx [T, H] from the sorted rows' gradients dxs [rows, H] (both of cfg.dtype)."""
    if elsewhere(dxs, stream):
        with on(dxs, stream):
            return sort_grad(cfg, dxs, pos, ws, out)
    t, dev = cfg.dtype, dxs.get_device()
    dxs_ptr, ld_s = mat(dxs, "dxs", (cfg.rows, cfg.H), t, dev)
    pos_ptr, _ = _pos_gate(cfg, pos, None, dev)
    ws_ptr = workspace_ptr(ws, 256, dev)
    dx, dx_ptr, ld = _mat_out(out, dxs, "out", (cfg.T, cfg.H), t, dev)
    rc = (_lib or lib()).moe_rows_sort_grad(cfg.c(ld, ld_s), dxs_ptr, pos_ptr, dx_ptr, ws_ptr, raw_stream(dev))
    if rc:
        raise moe.MoeError(rc, "moe_rows_sort_grad")
    return dx


def unsort_grad(cfg: Config, dy, ys, gate, pos, ws, out=None, dgate=None, stream=None):
    """(dys [rows, H] of slot_dtype, dgate fp32 [T, K]) from dy [T, H].  ``out`` may be ys itself; rows
    that no assignment holds are left as they were."""
    if elsewhere(dy, stream):
        with on(dy, stream):
            return unsort_grad(cfg, dy, ys, gate, pos, ws, out, dgate)
    slots, t, dev = (cfg.rows, cfg.H), cfg.slot_dtype, dy.get_device()
    dy_ptr, ld = mat(dy, "dy", (cfg.T, cfg.H), cfg.dtype, dev)
    ys_ptr, ld_s = mat(ys, "ys", slots, t, dev)
    pos_ptr, gate_ptr = _pos_gate(cfg, pos, gate, dev)
    ws_ptr = workspace_ptr(ws, 256, dev)
    dys, dys_ptr, ld_d = _mat_out(out, dy, "out", slots, t, dev)
    dgate, dgate_ptr = _vec_out(dgate, dy, "dgate", (cfg.T, cfg.K), torch.float32, dev)
    rc = (_lib or lib()).moe_rows_unsort_grad(cfg.c(ld, ld_s, 0, ld_d), dy_ptr, ys_ptr, gate_ptr, pos_ptr, dys_ptr,
                                              dgate_ptr, ws_ptr, raw_stream(dev))
    if rc:
        raise moe.MoeError(rc, "moe_rows_unsort_grad")
    return dys, dgate
