"""Thin ctypes binding of the 8-bit path in libsrm_moe.so (declared in
include/srm_q8.h): rows in 8 bits with one scale per row, with or without the
residual's addition and the RMSNorm, and products of 8-bit integers with a scale
per row and per channel, dense or by expert groups.

Argument marshalling only: every step runs in the library's CUDA kernels;
PyTorch supplies device memory and the current stream of the tensors' device.
No fallback: if the library is missing, every call raises.

    q, scale = q8.add_rmsnorm(x, gamma, delta=attn_out, x_out=x, y=x_ffn)
    q, scale = q8.quantize(h)
    h = q8.dequantize(q, scale, torch.float16)

    cfg = q8.MatmulConfig(R, N, K, dtype=torch.bfloat16)   # groups=, swiglu= for the experts
    ws = q8.workspace(cfg)
    y = q8.matmul(cfg, q, scale, w, w_scale, ws, residual=x)
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses

import torch

from . import moe

SYMBOLS = ("moe_q8_add_rmsnorm", "moe_q8_quantize", "moe_q8_dequantize", "moe_q8_pack_weights",
           "moe_q8_matmul_workspace_size", "moe_q8_matmul")

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3}


class _Rows(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("ld_x", ctypes.c_int64), ("ld_delta", ctypes.c_int64), ("ld_sum", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_q", ctypes.c_int64)]


class _Matmul(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("swiglu", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64), ("ld_residual", ctypes.c_int64)]


_bound = False


def lib():
    """The library with the 8-bit entry points typed."""
    global _bound
    L = moe.lib()
    if not _bound:
        vp, P = ctypes.c_void_p, ctypes.POINTER
        L.moe_q8_add_rmsnorm.restype = ctypes.c_int
        L.moe_q8_add_rmsnorm.argtypes = [P(_Rows), vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp]
        L.moe_q8_quantize.restype = ctypes.c_int
        L.moe_q8_quantize.argtypes = [P(_Rows), vp, vp, vp, vp]
        L.moe_q8_dequantize.restype = ctypes.c_int
        L.moe_q8_dequantize.argtypes = [P(_Rows), vp, vp, vp, vp]
        L.moe_q8_pack_weights.restype = ctypes.c_int
        L.moe_q8_pack_weights.argtypes = [P(moe._Cfg)] + [vp] * 11
        L.moe_q8_matmul_workspace_size.restype = ctypes.c_size_t
        L.moe_q8_matmul_workspace_size.argtypes = [P(_Matmul)]
        L.moe_q8_matmul.restype = ctypes.c_int
        L.moe_q8_matmul.argtypes = [P(_Matmul)] + [vp] * 8 + [ctypes.c_size_t, vp]
        _bound = True
    return L


# ------------------------------------------------------------------ marshalling

_NO_CONTEXT = contextlib.nullcontext()


def _on(device, stream):
    """Makes the tensors' device (and the call's stream, so that what the call
    allocates belongs to it) current for the call, where it is not already."""
    if stream is not None:
        if stream.device != device:
            raise ValueError("stream is on %s, the tensors are on %s" % (stream.device, device))
        return torch.cuda.stream(stream)
    return _NO_CONTEXT if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _rows(t, name, shape, dtypes, device=None):
    """A matrix [T, H] with contiguous rows, `shape` None or what it has to be."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a CUDA device" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the call on %s" % (name, t.device, device))
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(map(str, dtypes)), t.dtype))
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError("%s must have shape %s, got %s" % (name, shape or "[T, H]", tuple(t.shape)))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError("%s must have rows that do not overlap" % name)
    return t


def _vector(t, name, n, dtype, device):
    moe._req(t, dtype, (n,), name)
    if t.device != device:
        raise ValueError("%s is on %s, the call on %s" % (name, t.device, device))
    return t


def _ld(t):
    """Row stride in elements (a single row's is free, so the row length serves)."""
    return 0 if t is None else t.stride(0) if t.shape[0] > 1 else t.shape[1]


FLOATS = (torch.bfloat16, torch.float16, torch.float32)


def _q_out(out, T, H, device):
    if out is None:
        return (torch.empty((T, H), dtype=torch.int8, device=device),
                torch.empty((T,), dtype=torch.float32, device=device))
    q, scale = out
    _rows(q, "q", (T, H), (torch.int8,), device)
    _vector(scale, "scale", T, torch.float32, device)
    return q, scale


# ------------------------------------------------------------------ rows in 8 bits

def add_rmsnorm(x, gamma, eps=1e-5, delta=None, x_out=None, y=None, out=None, stream=None):
    """(q int8 [T, H], scale fp32 [T]) of the RMSNorm of x (+ delta).  x, delta: bf16, fp16 or fp32
    [T, H] with contiguous rows; gamma: [H] of the same type.  ``x_out`` receives x + delta and ``y``
    the normalised rows, both in x's type; each may be x or delta itself, but not the same one.
    ``out``: (q, scale) to write into."""
    _rows(x, "x", None, FLOATS)
    T, H, dev = x.shape[0], x.shape[1], x.device
    _vector(gamma, "gamma", H, x.dtype, dev)
    for t, name in ((delta, "delta"), (x_out, "x_out"), (y, "y")):
        if t is not None:
            _rows(t, name, (T, H), (x.dtype,), dev)
    with _on(dev, stream):
        q, scale = _q_out(out, T, H, dev)
        c = _Rows(T, H, DTYPES[x.dtype], _ld(x), _ld(delta), _ld(x_out), _ld(y), _ld(q))
        moe._check(lib().moe_q8_add_rmsnorm(ctypes.byref(c), moe._ptr(x), moe._ptr(delta), moe._ptr(gamma),
                                            float(eps), moe._ptr(x_out), moe._ptr(y), moe._ptr(q),
                                            moe._ptr(scale), moe._stream(stream)), "moe_q8_add_rmsnorm")
    return q, scale


def quantize(x, out=None, stream=None):
    """(q int8 [T, H], scale fp32 [T]): rows of x (bf16, fp16 or fp32) in 8 bits."""
    _rows(x, "x", None, FLOATS)
    T, H, dev = x.shape[0], x.shape[1], x.device
    with _on(dev, stream):
        q, scale = _q_out(out, T, H, dev)
        c = _Rows(T, H, DTYPES[x.dtype], _ld(x), 0, 0, 0, _ld(q))
        moe._check(lib().moe_q8_quantize(ctypes.byref(c), moe._ptr(x), moe._ptr(q), moe._ptr(scale),
                                         moe._stream(stream)), "moe_q8_quantize")
    return q, scale


def dequantize(q, scale, dtype=torch.bfloat16, out=None, stream=None):
    """The values q * scale as ``dtype`` (bf16, fp16 or fp32) [T, H]."""
    _rows(q, "q", None, (torch.int8,))
    T, H, dev = q.shape[0], q.shape[1], q.device
    _vector(scale, "scale", T, torch.float32, dev)
    if dtype not in FLOATS:
        raise TypeError("dtype must be %s, got %s" % (" or ".join(map(str, FLOATS)), dtype))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((T, H), dtype=dtype, device=dev)
        _rows(out, "out", (T, H), (dtype,), dev)
        c = _Rows(T, H, DTYPES[dtype], 0, 0, 0, _ld(out), _ld(q))
        moe._check(lib().moe_q8_dequantize(ctypes.byref(c), moe._ptr(q), moe._ptr(scale), moe._ptr(out),
                                           moe._stream(stream)), "moe_q8_dequantize")
    return out


def pack_weights(cfg: moe.Config, w1, w3, w2, ws1=None, ws3=None, ws2=None, stream=None):
    """Expert weights (bf16, as moe.pack_weights takes them) in 8 bits with a scale per output channel:
    (w13 int8 [G * 2I, H], its scales fp32 [G * 2I], w2 int8 [G * H, I], its scales fp32 [G * H]),
    G = E + has_shared groups, W1 and W3 interleaved in units of 16 + 16 rows."""
    E, I, H, bf = cfg.E, cfg.I, cfg.H, torch.bfloat16
    if E > 0:
        moe._req(w1, bf, (E, I, H), "w1")
        moe._req(w3, bf, (E, I, H), "w3")
        moe._req(w2, bf, (E, H, I), "w2")
    if cfg.has_shared:
        moe._req(ws1, bf, (I, H), "ws1")
        moe._req(ws3, bf, (I, H), "ws3")
        moe._req(ws2, bf, (H, I), "ws2")
    dev = (w1 if E > 0 else ws1).device
    G = E + int(bool(cfg.has_shared))
    with _on(dev, stream):
        w13 = torch.empty((G * 2 * I, H), dtype=torch.int8, device=dev)
        w13_scale = torch.empty((G * 2 * I,), dtype=torch.float32, device=dev)
        w2q = torch.empty((G * H, I), dtype=torch.int8, device=dev)
        w2_scale = torch.empty((G * H,), dtype=torch.float32, device=dev)
        moe._check(lib().moe_q8_pack_weights(ctypes.byref(cfg.c()), moe._ptr(w1), moe._ptr(w3), moe._ptr(w2),
                                             moe._ptr(ws1), moe._ptr(ws3), moe._ptr(ws2), moe._ptr(w13),
                                             moe._ptr(w13_scale), moe._ptr(w2q), moe._ptr(w2_scale),
                                             moe._stream(stream)), "moe_q8_pack_weights")
    return w13, w13_scale, w2q, w2_scale


# ------------------------------------------------------------------ products

@dataclasses.dataclass(frozen=True)
class MatmulConfig:
    """R rows of K elements times `groups` weight matrices of N channels; swiglu: the channels are units of
    16 gate and 16 up ones and the result silu(gate) * up has N / 2 columns; dtype of the result."""
    R: int
    N: int
    K: int
    groups: int = 1
    swiglu: bool = False
    dtype: torch.dtype = torch.bfloat16

    @property
    def columns(self) -> int:
        return self.N // 2 if self.swiglu else self.N

    def c(self, x=None, y=None, residual=None) -> _Matmul:
        return _Matmul(self.R, self.N, self.K, self.groups, int(bool(self.swiglu)), DTYPES.get(self.dtype, -1),
                       _ld(x), _ld(y), _ld(residual))


def workspace_bytes(cfg: MatmulConfig) -> int:
    n = lib().moe_q8_matmul_workspace_size(ctypes.byref(cfg.c()))
    if n == 0:
        raise moe.MoeError(2, "moe_q8_matmul_workspace_size")
    return int(n)


def workspace(cfg: MatmulConfig, device=None) -> torch.Tensor:
    """A workspace tensor (uint8), its control words zeroed."""
    ws = torch.empty(workspace_bytes(cfg), dtype=torch.uint8, device=device or "cuda")
    ws[:256].zero_()
    return ws


def matmul(cfg: MatmulConfig, x, x_scale, w, w_scale, ws, offsets=None, residual=None, out=None, stream=None):
    """y [R, N] (with swiglu [R, N / 2]) = x_scale * w_scale * (x . w) (+ residual).  x: int8 [R, K] with rows
    16-byte aligned; w: int8 [groups * N, K]; offsets: int32, at least groups + 1 entries (moe.permute's),
    or None with one group.  ``out`` may be the residual itself."""
    _rows(x, "x", (cfg.R, cfg.K), (torch.int8,))
    dev = x.device
    _vector(x_scale, "x_scale", cfg.R, torch.float32, dev)
    moe._req(w, torch.int8, (cfg.groups * cfg.N, cfg.K), "w")
    if w.device != dev:
        raise ValueError("w is on %s, the call on %s" % (w.device, dev))
    _vector(w_scale, "w_scale", cfg.groups * cfg.N, torch.float32, dev)
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < cfg.groups + 1:
            raise ValueError("offsets must have at least %d entries" % (cfg.groups + 1))
        _vector(offsets, "offsets", offsets.numel(), torch.int32, dev)
    if residual is not None:
        _rows(residual, "residual", (cfg.R, cfg.columns), (cfg.dtype,), dev)
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.device != dev:
        raise TypeError("ws must be a uint8 tensor on %s" % dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty((cfg.R, cfg.columns), dtype=cfg.dtype, device=dev)
        _rows(out, "out", (cfg.R, cfg.columns), (cfg.dtype,), dev)
        moe._check(lib().moe_q8_matmul(ctypes.byref(cfg.c(x, out, residual)), moe._ptr(x), moe._ptr(x_scale),
                                       moe._ptr(w), moe._ptr(w_scale), moe._ptr(offsets), moe._ptr(residual),
                                       moe._ptr(out), moe._ptr(ws), ws.numel(), moe._stream(stream)),
                   "moe_q8_matmul")
    return out
