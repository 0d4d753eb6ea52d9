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

import ctypes
import dataclasses

import torch

from . import moe
from .marshal import DTYPES, FLOATS, elsewhere, mat, on, raw_stream, rows_of, vec
from .marshal import workspace as workspace_ptr

SYMBOLS = ("moe_q8_add_rmsnorm", "moe_q8_quantize", "moe_q8_dequantize", "moe_q8_pack_weights",
           "moe_q8_matmul_workspace_size", "moe_q8_workspace_init", "moe_q8_matmul")


class _Rows(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("ld_x", ctypes.c_int64), ("ld_delta", ctypes.c_int64), ("ld_sum", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_q", ctypes.c_int64)]


class _Matmul(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("swiglu", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64), ("ld_residual", ctypes.c_int64)]


_lib = None


def lib():
    """The library with the 8-bit entry points typed."""
    global _lib
    if _lib is None:
        L = moe.lib()
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
        L.moe_q8_workspace_init.restype = ctypes.c_int
        L.moe_q8_workspace_init.argtypes = [vp, ctypes.c_size_t, vp]
        L.moe_q8_matmul.restype = ctypes.c_int
        L.moe_q8_matmul.argtypes = [P(_Matmul)] + [vp] * 8 + [ctypes.c_size_t, vp]
        _lib = L
    return _lib


# ------------------------------------------------------------------ rows in 8 bits

def _q_out(out, x, shape, dev):
    if out is None:
        q, scale = x.new_empty(shape, dtype=torch.int8), x.new_empty(shape[0], dtype=torch.float32)
        return q, q.data_ptr(), shape[1], scale, scale.data_ptr()
    q, scale = out
    q_ptr, ld_q = mat(q, "q", shape, torch.int8, dev)
    return q, q_ptr, ld_q, scale, vec(scale, "scale", shape[:1], torch.float32, dev)


def add_rmsnorm(x, gamma, eps=1e-5, delta=None, x_out=None, y=None, out=None, stream=None):
    """(q int8 [T, H], scale fp32 [T]) of the RMSNorm of x (+ delta).  x, delta: bf16, fp16 or fp32
    [T, H] with contiguous rows; gamma: [H] of the same type.  ``x_out`` receives x + delta and ``y``
    the normalised rows, both in x's type; each may be x or delta itself, but not the same one.
    ``out``: (q, scale) to write into."""
    if elsewhere(x, stream):
        with on(x, stream):
            return add_rmsnorm(x, gamma, eps, delta, x_out, y, out)
    shape, t, dev = rows_of(x, "x", FLOATS), x.dtype, x.get_device()
    x_ptr, ld = mat(x, "x", shape, t, dev)
    g_ptr = vec(gamma, "gamma", shape[1:], t, dev)
    d_ptr, ld_d = mat(delta, "delta", shape, t, dev) if delta is not None else (None, 0)
    s_ptr, ld_s = mat(x_out, "x_out", shape, t, dev) if x_out is not None else (None, 0)
    y_ptr, ld_y = mat(y, "y", shape, t, dev) if y is not None else (None, 0)
    q, q_ptr, ld_q, scale, scale_ptr = _q_out(out, x, shape, dev)
    c = _Rows(shape[0], shape[1], DTYPES[t], ld, ld_d, ld_s, ld_y, ld_q)
    rc = (_lib or lib()).moe_q8_add_rmsnorm(c, x_ptr, d_ptr, g_ptr, eps, s_ptr, y_ptr, q_ptr, scale_ptr, raw_stream(dev))
    if rc:
        raise moe.MoeError(rc, "moe_q8_add_rmsnorm")
    return q, scale


def quantize(x, out=None, stream=None):
    """(q int8 [T, H], scale fp32 [T]): rows of x (bf16, fp16 or fp32) in 8 bits."""
    if elsewhere(x, stream):
        with on(x, stream):
            return quantize(x, out)
    shape, t, dev = rows_of(x, "x", FLOATS), x.dtype, x.get_device()
    x_ptr, ld = mat(x, "x", shape, t, dev)
    q, q_ptr, ld_q, scale, scale_ptr = _q_out(out, x, shape, dev)
    rc = (_lib or lib()).moe_q8_quantize(_Rows(shape[0], shape[1], DTYPES[t], ld, 0, 0, 0, ld_q), x_ptr, q_ptr,
                                         scale_ptr, raw_stream(dev))
    if rc:
        raise moe.MoeError(rc, "moe_q8_quantize")
    return q, scale


def dequantize(q, scale, dtype=torch.bfloat16, out=None, stream=None):
    """The values q * scale as ``dtype`` (bf16, fp16 or fp32) [T, H]."""
    if elsewhere(q, stream):
        with on(q, stream):
            return dequantize(q, scale, dtype, out)
    shape, dev = rows_of(q, "q", (torch.int8,)), q.get_device()
    if dtype not in FLOATS:
        raise TypeError("dtype must be %s, got %s" % (" or ".join(map(str, FLOATS)), dtype))
    q_ptr, ld_q = mat(q, "q", shape, torch.int8, dev)
    scale_ptr = vec(scale, "scale", shape[:1], torch.float32, dev)
    if out is None:
        out = q.new_empty(shape, dtype=dtype)
        y_ptr, ld_y = out.data_ptr(), shape[1]
    else:
        y_ptr, ld_y = mat(out, "out", shape, dtype, dev)
    rc = (_lib or lib()).moe_q8_dequantize(_Rows(shape[0], shape[1], DTYPES[dtype], 0, 0, 0, ld_y, ld_q), q_ptr,
                                           scale_ptr, y_ptr, raw_stream(dev))
    if rc:
        raise moe.MoeError(rc, "moe_q8_dequantize")
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
    like = w1 if E > 0 else ws1
    G, dev = E + int(bool(cfg.has_shared)), like.device
    with on(like, stream):
        w13 = torch.empty((G * 2 * I, H), dtype=torch.int8, device=dev)
        w13_scale = torch.empty((G * 2 * I,), dtype=torch.float32, device=dev)
        w2q = torch.empty((G * H, I), dtype=torch.int8, device=dev)
        w2_scale = torch.empty((G * H,), dtype=torch.float32, device=dev)
        moe._check(lib().moe_q8_pack_weights(ctypes.byref(cfg.c()), moe._ptr(w1), moe._ptr(w3), moe._ptr(w2),
                                             moe._ptr(ws1), moe._ptr(ws3), moe._ptr(ws2), moe._ptr(w13),
                                             moe._ptr(w13_scale), moe._ptr(w2q), moe._ptr(w2_scale),
                                             raw_stream(like.get_device())), "moe_q8_pack_weights")
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

    def c(self) -> _Matmul:
        return _Matmul(self.R, self.N, self.K, self.groups, int(bool(self.swiglu)), DTYPES.get(self.dtype, -1),
                       self.K, self.columns, self.columns)


def workspace_bytes(cfg: MatmulConfig) -> int:
    n = lib().moe_q8_matmul_workspace_size(ctypes.byref(cfg.c()))
    if n == 0:
        raise moe.MoeError(2, "moe_q8_matmul_workspace_size")
    return int(n)


def workspace(*cfgs: MatmulConfig, device=None) -> torch.Tensor:
    """An initialised workspace tensor (uint8) that serves products of these shapes, one at a time."""
    ws = torch.empty(max(workspace_bytes(c) for c in cfgs), dtype=torch.uint8, device=device or "cuda")
    init_workspace(ws)
    return ws


def init_workspace(ws):
    """Sets a workspace's control words: once for memory allocated elsewhere, and after a call that
    reported MOE_ERR_TIMEOUT."""
    with on(ws, None):
        dev = ws.get_device()
        moe._check(lib().moe_q8_workspace_init(workspace_ptr(ws, 256, dev), ws.numel(), raw_stream(dev)),
                   "moe_q8_workspace_init")


def matmul(cfg: MatmulConfig, x, x_scale, w, w_scale, ws, offsets=None, residual=None, out=None, stream=None):
    """y [R, N] (with swiglu [R, N / 2]) = x_scale * w_scale * (x . w) (+ residual).  x: int8 [R, K] with rows
    16-byte aligned; w: int8 [groups * N, K]; offsets: int32, at least groups + 1 entries (moe.permute's),
    or None with one group.  ``out`` may be the residual itself."""
    if elsewhere(x, stream):
        with on(x, stream):
            return matmul(cfg, x, x_scale, w, w_scale, ws, offsets, residual, out)
    R, N, K, G, t, dev = cfg.R, cfg.N, cfg.K, cfg.groups, cfg.dtype, x.get_device()
    shape = (R, N // 2 if cfg.swiglu else N)
    x_ptr, ld_x = mat(x, "x", (R, K), torch.int8, dev)
    xs_ptr = vec(x_scale, "x_scale", (R,), torch.float32, dev)
    w_ptr = vec(w, "w", (G * N, K), torch.int8, dev)
    ws_ptr = vec(w_scale, "w_scale", (G * N,), torch.float32, dev)
    off_ptr = None
    if offsets is not None:
        if offsets.dim() != 1 or offsets.shape[0] < G + 1:
            raise ValueError("offsets must have at least %d entries" % (G + 1))
        off_ptr = vec(offsets, "offsets", offsets.shape, torch.int32, dev)
    r_ptr, ld_r = mat(residual, "residual", shape, t, dev) if residual is not None else (None, 0)
    work = workspace_ptr(ws, 256, dev)
    if out is None:
        out = x.new_empty(shape, dtype=t)
        y_ptr, ld_y = out.data_ptr(), shape[1]
    else:
        y_ptr, ld_y = mat(out, "out", shape, t, dev)
    c = _Matmul(R, N, K, G, 1 if cfg.swiglu else 0, DTYPES.get(t, -1), ld_x, ld_y, ld_r)
    rc = (_lib or lib()).moe_q8_matmul(c, x_ptr, xs_ptr, w_ptr, ws_ptr, off_ptr, r_ptr, y_ptr, work, ws.numel(),
                                       raw_stream(dev))
    if rc:
        raise moe.MoeError(rc, "moe_q8_matmul")
    return out


# ------------------------------------------------------------------ blocks

class MoeBlock:
    """One MoE block in 8 bits: ``y = block(x)``, the 8-bit form of moe.MoeBlock (same arguments).

    Router and selection are the bf16 block's; the experts' products take 8-bit rows and weights, the
    rows go to the experts in 8 bits (half the bytes) and come back with the gates applied by the row
    calls.  Its buffers belong to the block: one call at a time, and y holds until the next."""

    def __init__(self, cfg: moe.Config, w_router, bias, w1, w3, w2, ws1=None, ws3=None, ws2=None, packed=None):
        from . import ep, rows  # rows shares this module's marshalling
        self._rows = rows
        self.cfg, self.w_router, self.bias = cfg, w_router, bias
        # packed: pack_weights' result for this block's H, I and E, shared with another block
        self.weights = packed if packed is not None else pack_weights(cfg, w1, w3, w2, ws1, ws3, ws2)
        self.router_packed = moe.pack_router(cfg, w_router)
        dev, T, K, E, H, I, P = w_router.device, cfg.T, cfg.K, cfg.E, cfg.H, cfg.I, cfg.rows
        self.ws = moe.workspace(cfg, device=dev)
        G = E + int(bool(cfg.has_shared))
        self.up = MatmulConfig(P, 2 * I, H, groups=G, swiglu=True, dtype=torch.float16)
        self.down = MatmulConfig(P, H, I, groups=G, dtype=torch.float16)
        self.mm_ws = workspace(self.up, self.down, device=dev)
        self.there = rows.Config.of(cfg, dtype=torch.int8)
        self.back = rows.Config.of(cfg)
        self.idx = torch.empty((T, K), dtype=torch.int32, device=dev)
        self.gate = torch.empty((T, K), dtype=torch.float32, device=dev)
        self.margin = torch.empty((T,), dtype=torch.float32, device=dev)
        self.counts = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        self.offsets = torch.empty((E + 2,), dtype=torch.int32, device=dev)
        self.sorted = torch.empty((P,), dtype=torch.int32, device=dev)
        self.pos = torch.empty((P,), dtype=torch.int32, device=dev)
        self.q = (torch.empty((T, H), dtype=torch.int8, device=dev), torch.empty((T,), dtype=torch.float32, device=dev))
        # the sorted rows and the experts' outputs use the places the bf16 block's workspace has for them
        at = ep.workspace_offset(cfg, ep.WS_TOKEN_ROWS) if T else 0
        self.xs = self.ws[at:at + P * H].view(torch.int8).view(P, H)
        self.xs_scale = torch.empty((P,), dtype=torch.float32, device=dev)
        self.h = torch.empty((P, I), dtype=torch.float16, device=dev)
        self.hq = (torch.empty((P, I), dtype=torch.int8, device=dev), torch.empty((P,), dtype=torch.float32, device=dev))
        at = ep.workspace_offset(cfg, ep.WS_SLOT_OUTPUTS) if T else 0
        self.ys = self.ws[at:at + 2 * P * H].view(torch.float16).view(P, H)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)

    def _run(self, x_ffn, residual, logits):
        w13, w13_scale, w2, w2_scale = self.weights
        rows = self._rows
        moe.route_packed(self.cfg, x_ffn, self.router_packed, self.bias, self.ws,
                         out=(self.idx, self.gate, self.margin), logits=logits)
        moe.permute(self.cfg, self.idx, self.ws, out=(self.counts, self.offsets, self.sorted))
        rows.sort(self.there, self.q[0], self.offsets, self.sorted, self.ws, x_scale=self.q[1], out=self.xs,
                  pos=self.pos, xs_scale=self.xs_scale)
        matmul(self.up, self.xs, self.xs_scale, w13, w13_scale, self.mm_ws, offsets=self.offsets, out=self.h)
        quantize(self.h, out=self.hq)
        matmul(self.down, self.hq[0], self.hq[1], w2, w2_scale, self.mm_ws, offsets=self.offsets, out=self.ys)
        return rows.unsort(self.back, self.ys, self.gate, self.pos, self.ws, residual=residual, out=self.y)

    def sublayer(self, x_resid, gamma, eps=1e-5, stream=None, logits=None, delta=None):
        """The decoder block's FFN sublayer: x' + MoE(RMSNorm(x')) and the normalised rows, with
        x' = x_resid + delta in one pass where the previous sublayer's output ``delta`` is given."""
        if elsewhere(x_resid, stream):
            with on(x_resid, stream):
                return self.sublayer(x_resid, gamma, eps, None, logits, delta)
        x_ffn = torch.empty_like(x_resid)
        x_sum = x_resid if delta is None else torch.empty_like(x_resid)
        add_rmsnorm(x_resid, gamma, eps, delta=delta, x_out=None if delta is None else x_sum, y=x_ffn, out=self.q)
        return self._run(x_ffn, x_sum, logits), x_ffn

    def __call__(self, x, stream=None, logits=None):
        if elsewhere(x, stream):
            with on(x, stream):
                return self(x, None, logits)
        quantize(x, out=self.q)
        return self._run(x, None, logits)

    def device_error(self, stream=None) -> int:
        """Read and clear the block's device error words (synchronises the stream)."""
        first, second = moe.device_error(self.ws, stream), moe.device_error(self.mm_ws, stream)
        return first or second


class DenseMlp:
    """A dense SwiGLU MLP in 8 bits (the 8-bit form of moe.dense_mlp): ``y = mlp(x)`` for up to cfg.T
    rows, cfg from moe.Config.dense; w1, w3: bf16 [I, H], w2: bf16 [H, I]."""

    def __init__(self, cfg: moe.Config, w1, w3, w2, packed=None):
        if cfg.E != 0 or cfg.K != 0 or not cfg.has_shared:
            raise ValueError("DenseMlp takes a moe.Config.dense configuration")
        self.cfg, self.dev = cfg, (packed[0] if packed is not None else w1).device
        self.weights = packed if packed is not None else pack_weights(cfg, None, None, None, w1, w3, w2)
        self.ws = workspace(*self._shapes(cfg.T), device=self.dev)

    def _shapes(self, R):
        H, I = self.cfg.H, self.cfg.I
        return MatmulConfig(R, 2 * I, H, swiglu=True, dtype=torch.float16), MatmulConfig(R, H, I)

    def __call__(self, x, residual=None, out=None, stream=None):
        """(residual +) W2 (silu(W1 x) * W3 x): bf16 [R, H], R <= cfg.T."""
        if elsewhere(x, stream):
            with on(x, stream):
                return self(x, residual, out)
        return self._mlp(quantize(x), residual, out)

    def sublayer(self, x_resid, gamma, eps=1e-5, delta=None, stream=None):
        """x' + MLP(RMSNorm(x')), x' = x_resid (+ delta)."""
        if elsewhere(x_resid, stream):
            with on(x_resid, stream):
                return self.sublayer(x_resid, gamma, eps, delta)
        x_sum = x_resid if delta is None else torch.empty_like(x_resid)
        q = add_rmsnorm(x_resid, gamma, eps, delta=delta, x_out=None if delta is None else x_sum)
        return self._mlp(q, x_sum, None)

    def _mlp(self, q, residual, out):
        w13, w13_scale, w2, w2_scale = self.weights
        R = q[0].shape[0]
        if R > self.cfg.T:
            raise ValueError("%d rows, the MLP was made for %d" % (R, self.cfg.T))
        up, down = self._shapes(R)
        h = matmul(up, q[0], q[1], w13, w13_scale, self.ws)
        hq, h_scale = quantize(h)
        return matmul(down, hq, h_scale, w2, w2_scale, self.ws, residual=residual, out=out)

    def device_error(self, stream=None) -> int:
        """Read and clear the device error word (synchronises the stream)."""
        return moe.device_error(self.ws, stream)
