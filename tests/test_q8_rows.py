"""Rows in 8 bits (include/srm_q8.h): the residual's addition, the RMSNorm and the quantisation against the
definition in 64 bits, and the refusals.

Tolerances.  u = 2^-24 is fp32's half step.  A row's sum of squares is a chain of at most m additions (the elements a
thread holds, then ten shuffle and warp steps), so the mean is off by at most (m + 2) u relative, its root by half that
plus the root's, the quotient's and two products' roundings: n is within c = (m / 2 + 6) u of the exact n, relative.
  scale: c + 2 u (the maximum's error and one division);  y: c and half a step of its type;
  q: the exact n / scale is at most 127 and off by 127 (2 c + 4 u) in the kernel's arithmetic, then rounded: 0.5 more."""
import ctypes

import pytest
import torch

from sigmoid_routed_mixture_b200 import moe, q8

U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


# ------------------------------------------------------------------ refusals (CPU)

def rows_cfg(T=4, H=64, dtype=0, ld=None):
    ld = H if ld is None else ld
    return q8._Rows(T, H, dtype, ld, ld, ld, ld, ld)


A = ctypes.c_void_p(0x100000)  # aligned; never dereferenced, validation fails first
B2 = ctypes.c_void_p(0x300000)
ODD = ctypes.c_void_p(0x100001)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(dtype=3), 1), (dict(dtype=7), 1), (dict(H=(1 << 20) + 1), 2),
    (dict(T=1 << 31), 2), (dict(ld=63), 1), (dict(ld=(1 << 40) + 1), 1),
])
def test_row_shapes_refused(kw, code):
    L = q8.lib()
    c = rows_cfg(**kw)
    assert L.moe_q8_add_rmsnorm(ctypes.byref(c), A, A, A, 1e-5, A, None, A, A, None) == code
    assert L.moe_q8_quantize(ctypes.byref(c), A, A, A, None) == code
    assert L.moe_q8_dequantize(ctypes.byref(c), A, A, A, None) == code


def test_row_pointers_refused():
    L = q8.lib()
    c = ctypes.byref(rows_cfg())
    assert L.moe_q8_add_rmsnorm(None, A, A, A, 1e-5, A, None, A, A, None) == 1
    assert L.moe_q8_add_rmsnorm(c, None, A, A, 1e-5, A, None, A, A, None) == 1
    assert L.moe_q8_add_rmsnorm(c, A, A, None, 1e-5, A, None, A, A, None) == 1
    assert L.moe_q8_add_rmsnorm(c, A, A, A, -1e-5, A, None, A, A, None) == 1
    assert L.moe_q8_add_rmsnorm(c, A, A, A, float("nan"), A, None, A, A, None) == 1
    assert L.moe_q8_add_rmsnorm(c, A, A, A, 1e-5, B2, B2, A, A, None) == 1  # sum and norm in one place
    apart = rows_cfg()
    apart.ld_y = 72  # a result in an input's place, its rows elsewhere
    assert L.moe_q8_add_rmsnorm(ctypes.byref(apart), A, B2, A, 1e-5, None, A, B2, B2, None) == 1
    assert L.moe_q8_add_rmsnorm(ctypes.byref(apart), B2, A, A, 1e-5, None, A, B2, B2, None) == 1
    apart.ld_sum = 72
    assert L.moe_q8_add_rmsnorm(ctypes.byref(apart), A, B2, A, 1e-5, A, None, B2, B2, None) == 1
    assert L.moe_q8_add_rmsnorm(c, ODD, A, A, 1e-5, A, None, A, A, None) == 3
    assert L.moe_q8_add_rmsnorm(c, A, A, A, 1e-5, A, ODD, A, A, None) == 3
    assert L.moe_q8_add_rmsnorm(c, A, A, A, 1e-5, A, None, A, ODD, None) == 3
    assert L.moe_q8_quantize(c, A, None, A, None) == 1
    assert L.moe_q8_quantize(c, ODD, A, A, None) == 3
    assert L.moe_q8_dequantize(c, A, None, A, None) == 1
    assert L.moe_q8_dequantize(c, A, A, ODD, None) == 3
    empty = ctypes.byref(rows_cfg(T=0))
    assert L.moe_q8_add_rmsnorm(empty, None, None, None, 1e-5, None, None, None, None, None) == 0
    assert L.moe_q8_quantize(empty, None, None, None, None) == 0
    assert L.moe_q8_dequantize(empty, None, None, None, None) == 0


def test_pack_refused():
    L = q8.lib()
    c = moe.Config(T=1, H=256, I=128, E=4, K=2).c()
    assert L.moe_q8_pack_weights(ctypes.byref(c), A, A, A, A, A, None, A, A, A, A, None) == 1
    assert L.moe_q8_pack_weights(ctypes.byref(c), A, A, A, A, A, A, A, A, ODD, A, None) == 3
    assert L.moe_q8_pack_weights(ctypes.byref(c), A, A, A, A, A, A, A, ODD, A, A, None) == 3
    assert L.moe_q8_pack_weights(None, A, A, A, A, A, A, A, A, A, A, None) == 1
    bad = moe.Config(T=1, H=200, I=128, E=4, K=2).c()
    assert L.moe_q8_pack_weights(ctypes.byref(bad), A, A, A, A, A, A, A, A, A, A, None) == 2


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        q8.quantize(x)
    with pytest.raises(TypeError):
        q8.quantize([1.0])


# ------------------------------------------------------------------ on the GPU

def chain(x):
    """The longest chain of fp32 additions of the kernel that takes these rows (at most)."""
    return max(32, -(-x.shape[1] // 1024)) + 10


def rows(T, H, dtype, seed, ld=None, offset=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ld = H if ld is None else ld
    base = torch.randn(T * ld + offset, generator=g, device="cuda").to(dtype)
    return base[offset:].as_strided((T, H), (ld, 1), offset)


def reference(x, gamma, eps, delta=None):
    total = x.double()
    if delta is not None:
        total = (x.double() + delta.double()).to(x.dtype).double()  # one rounding: both addends are exact in 64 bits
    n = total
    if gamma is not None:
        n = total / torch.sqrt((total * total).mean(1, keepdim=True) + eps) * gamma.double()
    return total.to(x.dtype), n


def check(x, n, q, scale, y=None, normed=True):
    c = (chain(x) / 2 + 6) * U if normed else 0.0
    s = n.abs().amax(1) / 127
    tiny = 2.0 ** -149
    assert torch.all((scale.double() - s).abs() <= (c + 2 * U) * s + tiny)
    ratio = torch.where(s[:, None] > 0, n / s[:, None], torch.zeros_like(n))
    off = (q.double() - ratio).abs()
    assert off.max().item() <= 0.5 + 127 * (2 * c + 4 * U)
    assert q.abs().max().item() <= 127
    if y is not None:
        half = torch.finfo(x.dtype).eps / 2
        smallest = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps
        assert torch.all((y.double() - n).abs() <= (c + half * (1 + c)) * n.abs() + smallest)


SHAPES = [(1, 1), (1, 6144), (3, 64), (5, 257), (7, 1541), (2, 4097), (300, 2048), (301, 1000), (1000, 8), (2, 40008),
          (400, 6144), (2, 9311), (3, 16391), (2, 30000), (301, 4097)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_add_rmsnorm(T, H, dtype):
    x, delta = rows(T, H, dtype, 1), rows(T, H, dtype, 2)
    gamma = (1 + 0.1 * rows(1, H, torch.float32, 3)[0]).to(dtype)
    total, y = torch.empty_like(x), torch.empty_like(x)
    q, scale = q8.add_rmsnorm(x, gamma, 1e-5, delta=delta, x_out=total, y=y)
    want, n = reference(x, gamma, 1e-5, delta)
    assert torch.equal(total, want)
    check(x, n, q, scale, y)
    again, scale2 = q8.add_rmsnorm(x, gamma, 1e-5, delta=delta)
    assert torch.equal(again, q) and torch.equal(scale2, scale)
    q, scale = q8.add_rmsnorm(x, gamma, 1e-5, x_out=total, y=y)  # without a delta the sum is x
    assert torch.equal(total, x)
    check(x, reference(x, gamma, 1e-5)[1], q, scale, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_quantize_and_back(T, H, dtype):
    x = rows(T, H, dtype, 4)
    q, scale = q8.quantize(x)
    check(x, x.double(), q, scale, normed=False)
    for out in DTYPES:
        v = q8.dequantize(q, scale, out)
        exact = q.double() * scale.double()[:, None]
        assert torch.all((v.double() - exact).abs() <= (torch.finfo(out).eps / 2 + 2 * U) * exact.abs() +
                         torch.finfo(out).smallest_normal * torch.finfo(out).eps)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ld,offset", [(72, 0), (67, 0), (72, 3), (64, 8)])
def test_strides_and_in_place(dtype, ld, offset):
    T, H = 33, 64
    x, delta = rows(T, H, dtype, 5, ld, offset), rows(T, H, dtype, 6, 80, 1)
    gamma = rows(1, H, dtype, 7)[0]
    want, n = reference(x, gamma, 1e-6, delta)
    qbuf = torch.full((T, ld + 5), 99, dtype=torch.int8, device="cuda")
    sc = torch.empty(T, dtype=torch.float32, device="cuda")
    # the stream's buffer takes the sum, the sublayer's output buffer the norm
    q, scale = q8.add_rmsnorm(x, gamma, 1e-6, delta=delta, x_out=x, y=delta, out=(qbuf[:, 2:2 + H], sc))
    assert torch.equal(x, want)
    check(x, n, q, scale, delta)
    assert bool((qbuf[:, :2] == 99).all()) and bool((qbuf[:, 2 + H:] == 99).all())
    y = q8.dequantize(q, scale, dtype, out=x)  # strided output
    assert torch.equal(y, q8.dequantize(q.contiguous(), scale, dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,ld", [(37, 61, 67), (300, 1541, 1541), (2000, 513, 515), (9, 3, 5), (11, 1, 3), (4, 4099, 4109),
                                    (700, 4099, 4099), (3, 16000, 16007), (6000, 257, 257)])
def test_rows_at_any_element(T, H, ld, dtype):
    """Aligned buffers whose rows start at any element, results in place: nothing beside the rows is touched."""
    def buffer(seed, kind):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        return torch.randn(T * ld, generator=g, device="cuda").to(kind).view(T, ld)

    xb, db, qb = buffer(20, dtype), buffer(21, dtype), torch.full((T, ld), 99, dtype=torch.int8, device="cuda")
    x, delta, q8b = xb[:, :H], db[:, :H], qb[:, :H]
    beside = [b[:, H:].clone() for b in (xb, db, qb)]
    gamma = (1 + 0.1 * rows(1, H, torch.float32, 22)[0]).to(dtype)
    sc = torch.empty(T, dtype=torch.float32, device="cuda")
    total, n = reference(x, gamma, 1e-5, delta)
    q, scale = q8.add_rmsnorm(x, gamma, 1e-5, delta=delta, x_out=x, y=delta, out=(q8b, sc))
    assert torch.equal(x, total)
    check(x, n, q, scale, delta)
    assert all(torch.equal(b[:, H:], w) for b, w in zip((xb, db, qb), beside))
    q, scale = q8.quantize(x, out=(q8b, sc))
    check(x, x.double(), q, scale, normed=False)
    want = q8.dequantize(q.contiguous(), scale, dtype)
    assert torch.equal(q8.dequantize(q, scale, dtype, out=x), want)
    exact = q.double() * scale.double()[:, None]
    assert torch.all((x.double() - exact).abs() <= (torch.finfo(dtype).eps / 2 + 2 * U) * exact.abs() +
                     torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps)
    assert all(torch.equal(b[:, H:], w) for b, w in zip((xb, db, qb), beside))


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 37, 2048, 40001])
def test_special_rows(H):
    dt = torch.float32
    x = rows(8, H, dt, 8)
    x[0] = 0
    x[1, H // 2] = float("inf")
    x[2, H - 1] = float("nan")
    x[3] *= 1e30   # squares overflow fp32
    x[4] *= 1e-30  # squares vanish beside eps
    x[5, 0] = float("-inf")
    x[6] = 3e38
    gamma = torch.ones(H, device="cuda")
    q, scale = q8.add_rmsnorm(x, gamma, 1e-5)
    assert scale[0].item() == 0 and not q[0].any()
    for r in (1, 2, 5):
        assert torch.isnan(scale[r]) and not q[r].any()
    fine = [3, 4, 6, 7]
    n = reference(x[fine], gamma, 1e-5)[1]
    check(x[fine], n, q[fine], scale[fine])
    # eps 0: tiny rows are scaled like any other
    n = reference(x[fine], gamma, 0.0)[1]
    q, scale = q8.add_rmsnorm(x[fine], gamma, 0.0)
    check(x[fine], n, q, scale)
    # quantisation alone, down to rows of subnormal scale
    for f in (1.0, 1e-20, 1e-37):
        v = rows(4, H, dt, 9) * f
        q, scale = q8.quantize(v)
        check(v, v.double(), q, scale, normed=False)
    q, scale = q8.quantize(x)
    assert scale[0].item() == 0 and torch.isnan(scale[[1, 2, 5]]).all() and not q[[0, 1, 2, 5]].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,most,H,power", [
    (torch.float16, 2047, 2048, 0), (torch.float16, 2047, 2049, -10), (torch.bfloat16, 255, 256, 100),
    (torch.bfloat16, 255, 40001, -100), (torch.float32, 2047, 2048, 115), (torch.float32, 2047, 2055, -130),
])
def test_ties_go_to_even(dtype, most, H, power):
    """Rows of the integers 0 .. M (times a power of two, signs mixed) for every M: 127 n / M is exactly k + 1/2 in
    many places, and elsewhere at least 1 / (2 M) away from it.  Equality, against integer arithmetic."""
    M = torch.arange(1, most + 1, dtype=torch.int64, device="cuda")[:, None]
    n = torch.minimum(torch.arange(H, dtype=torch.int64, device="cuda")[None], M)
    q2 = 254 * n + M  # twice M times (the quotient + 1/2)
    want = q2 // (2 * M)
    tie = q2 % (2 * M) == 0
    assert int(tie.sum()) > 200  # 253 for M up to 255
    want -= (tie & (want % 2 == 1)).long()
    sign = 1 - 2 * ((n + M) % 3 == 0).long()
    x = (n * sign).double() * 2.0 ** power
    assert torch.equal(x.to(dtype).double(), x)
    q, scale = q8.quantize(x.to(dtype))
    assert torch.equal(q.long(), want * sign)
    q = q8.quantize(x.to(dtype)[:, : most // 2 + 1])[0]  # rows of fewer threads; M above it gives another maximum
    cut = M[:, 0] <= most // 2
    assert torch.equal(q.long()[cut], (want * sign)[cut, : most // 2 + 1])


@pytest.mark.gpu
def test_other_stream_capture_and_empty():
    x, gamma = rows(64, 512, torch.bfloat16, 10), rows(1, 512, torch.bfloat16, 11)[0]
    want = q8.add_rmsnorm(x, gamma)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, scale = q8.add_rmsnorm(x, gamma, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(q, want[0]) and torch.equal(scale, want[1])
    out = (torch.empty_like(q), torch.empty_like(scale))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8.add_rmsnorm(x, gamma, out=out)
    x.mul_(2)
    x[3] = 0
    graph.replay()
    now = q8.add_rmsnorm(x, gamma)
    assert torch.equal(out[0], now[0]) and torch.equal(out[1], now[1]) and not out[0][3].any()
    q, scale = q8.quantize(x[:0])
    assert q.shape == (0, 512) and scale.shape == (0,)


@pytest.mark.gpu
def test_binding_refusals():
    x = rows(4, 64, torch.bfloat16, 12)
    gamma = x[0].clone()
    with pytest.raises(ValueError):
        q8.add_rmsnorm(x, gamma[:32])
    with pytest.raises(TypeError):
        q8.add_rmsnorm(x, gamma.float())
    with pytest.raises(ValueError, match="contiguous"):
        q8.quantize(x.t())
    with pytest.raises(ValueError, match="overlap"):
        q8.quantize(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        q8.add_rmsnorm(x, gamma, delta=x[:2])
    with pytest.raises(moe.MoeError):
        y = torch.empty_like(x)
        q8.add_rmsnorm(x, gamma, x_out=y, y=y)
    with pytest.raises(TypeError):
        q8.dequantize(x.to(torch.int8), x[:, 0].float(), torch.float64)


@pytest.mark.gpu
@pytest.mark.parametrize("E,shared", [(3, True), (2, False), (0, True)])
def test_pack_weights(E, shared):
    H, I = 256, 128
    cfg = moe.Config(T=1, H=H, I=I, E=E, K=min(E, 2), has_shared=shared)
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").mul_(0.02).to(torch.bfloat16)  # noqa: E731
    w1, w3, w2 = draw(E, I, H), draw(E, I, H), draw(E, H, I)
    ws = (draw(I, H), draw(I, H), draw(H, I)) if shared else (None, None, None)
    w13, s13, w2q, s2 = q8.pack_weights(cfg, w1, w3, w2, *ws)
    ups = torch.cat([w1, ws[0][None]]) if shared else w1
    gates = torch.cat([w3, ws[1][None]]) if shared else w3
    downs = torch.cat([w2, ws[2][None]]) if shared else w2
    G = downs.shape[0]
    units = torch.stack([ups.view(G, I // 16, 16, H), gates.view(G, I // 16, 16, H)], 2).reshape(G * 2 * I, H)
    for got, scale, w in ((w13, s13, units), (w2q, s2, downs.reshape(G * H, I))):
        q, s = q8.quantize(w)
        assert torch.equal(got, q) and torch.equal(scale, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,top,power", [(torch.bfloat16, 255, 0), (torch.float16, 2047, -12), (torch.bfloat16, 255, 90),
                                             (torch.bfloat16, 255, -100)])
@pytest.mark.parametrize("T,H", [(20000, 256), (3000, 2048), (200, 6144), (2500, 2047), (2500, 385), (150, 16391), (60, 40001)])
def test_norm_rounds_every_quotient(T, H, dtype, top, power):
    """n / scale does not depend on the root that n is divided by: of 16-bit rows it is 127 u / max |u| with u the exact
    product of x and gamma.  Whole x and gamma times powers of two, equality against integer arithmetic; ties to even."""
    g = torch.Generator(device="cuda")
    g.manual_seed(30)
    a = (torch.randn(T, H, generator=g, device="cuda") * top / 4).round().clamp(-top, top)
    b = torch.randint(top // 2, top + 1, (H,), generator=g, device="cuda")
    less = torch.arange(H, device="cuda") % 5
    exact = a.double() * torch.tensor([2.0 ** (power - k) for k in range(5)], dtype=torch.float64, device="cuda")[less]
    x, gamma = exact.to(dtype), (b.double() / (top + 1)).to(dtype)
    assert torch.equal(x.double(), exact) and torch.equal(gamma.double() * (top + 1), b.double())
    q, scale = q8.add_rmsnorm(x, gamma, 0.0)
    u = a.long() * b * 2 ** (4 - less)
    M = u.abs().amax(1, keepdim=True)
    twice = 254 * u.abs() + M  # twice M times (the quotient + 1/2)
    want = twice // (2 * M)
    want -= ((twice % (2 * M) == 0) & (want % 2 == 1)).long()
    assert torch.equal(q.long(), want * u.sign())
    check(x, reference(x, gamma, 0.0)[1], q, scale)
