"""Products of 8-bit integers with scales (include/srm_q8.h) against the definition in 64 bits, and the refusals.

Tolerances.  u = 2^-24 is fp32's half step, e half a step of the result's type.  The sum is an exact integer; its
conversion, the two scales and the residual's addition round once each: 3 u |v| + u (|v| + |r|) before the last
rounding.  silu(g) up: g and up are off by 3 u each, silu magnifies g's relative error by at most 1 + |g|; the
exponential is off by its argument's rounding, at most 2 |g| u, and the approximations' 2^-21 (results of 16 bits) or
8 u (fp32): (14 + 6 |g|) u + 2^-21 together.  The approximate reciprocal drops sigmoids below 2^-126."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from sigmoid_routed_mixture_b200 import moe, q8

U = 2.0 ** -24
DT = [torch.bfloat16, torch.float16, torch.float32]
A = ctypes.c_void_p(0x100000)  # aligned; never dereferenced, validation fails first
ODD = ctypes.c_void_p(0x100008)


# ------------------------------------------------------------------ refusals (CPU)

def c_cfg(R=5, N=64, K=64, groups=1, swiglu=0, dtype=0, ld_x=None, ld_y=None, ld_r=None):
    return q8._Matmul(R, N, K, groups, swiglu, dtype, ld_x or K, ld_y or N, ld_r or N)


def call(c, x=A, xs=A, w=A, ws_=A, off=A, res=None, y=A, ws=A, n=1 << 40):
    return q8.lib().moe_q8_matmul(ctypes.byref(c), x, xs, w, ws_, off, res, y, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(groups=0), 1), (dict(swiglu=2), 1), (dict(dtype=3), 1),
    (dict(K=72), 2), (dict(K=65552), 2), (dict(swiglu=1, N=48), 2), (dict(groups=258), 2), (dict(R=1 << 31), 2),
    (dict(groups=200, N=1 << 24), 2),
])
def test_shapes_refused(kw, code):
    c = c_cfg(**kw)
    assert call(c) == code
    assert q8.lib().moe_q8_matmul_workspace_size(ctypes.byref(c)) == 0


def test_pointers_refused():
    c = c_cfg()
    for bad in ("x", "xs", "w", "ws_", "y", "ws"):
        assert call(c, **{bad: None}) == 1, bad
    for bad in ("x", "w", "ws"):
        assert call(c, **{bad: ODD}) == 3, bad
    odd = ctypes.c_void_p(0x100001)
    for bad in ("xs", "ws_", "off", "y", "res"):
        assert call(c, **{bad: odd}) == 3, bad
    assert call(c_cfg(ld_x=72)) == 3  # rows off 16 bytes
    assert call(c_cfg(ld_x=48)) == 1 and call(c_cfg(ld_y=63)) == 1 and call(c_cfg(ld_r=63), res=A) == 1
    assert call(c_cfg(ld_r=72), res=A) == 1  # in place, its rows elsewhere
    assert call(c_cfg(groups=2), off=None) == 1
    assert call(c_cfg(swiglu=1), res=A) == 1
    need = q8.lib().moe_q8_matmul_workspace_size(ctypes.byref(c))
    assert call(c, n=need - 1) == 4
    assert call(c_cfg(R=0), **{k: None for k in ("x", "xs", "w", "ws_", "off", "y", "ws")}) == 0
    init = q8.lib().moe_q8_workspace_init
    assert init(None, 1 << 20, None) == 1 and init(ODD, 1 << 20, None) == 3 and init(A, 256, None) == 4
    assert q8.lib().moe_q8_matmul(None, A, A, A, A, A, None, A, A, 1 << 40, None) == 1


@pytest.mark.parametrize("groups,N", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 127), (1, 2 ** 31 - 255), (2, 2 ** 30 - 1),
                                      (257, (2 ** 31 - 1) // 257)])
def test_channels_whose_tiles_pass_31_bits_refused(groups, N):
    """The last tile's end has to be a 32-bit number: N + 127 wrapped, there were no tiles, and y was not written."""
    c = c_cfg(R=3, N=N, K=16, groups=groups)
    assert q8.lib().moe_q8_matmul_workspace_size(ctypes.byref(c)) == 0
    assert call(c) == 2
    most = (2 ** 31 - 256) // groups
    assert q8.lib().moe_q8_matmul_workspace_size(ctypes.byref(c_cfg(R=3, N=most, K=16, groups=groups))) > 0


def test_headers_are_plain_c(tmp_path):
    src = tmp_path / "client.c"
    src.write_text('#include "srm_rows.h"\n#include "srm_q8.h"\n'
                   "int main(void) { moe_q8_matmul_t c = {1, 32, 16, 1, 0, MOE_DTYPE_BF16, 16, 32, 32};\n"
                   "moe_rows_cfg_t r = {0};\n"
                   "return (moe_q8_matmul_workspace_size(&c) > 0 && moe_rows_sort_grad(&r, 0, 0, 0, 0, 0) == MOE_ERR_ARG)"
                   " ? 0 : 1; }\n")
    lib_dir, exe = os.path.dirname(moe.LIB_PATH), tmp_path / "client"
    inc = os.path.join(os.path.dirname(lib_dir), "include")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", inc, str(src), "-L", lib_dir, "-lsrm_moe",
                    "-Wl,-rpath," + lib_dir, "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_arrivals_on_another_cta_have_cluster_scope():
    """mbarrier.arrive on a shared::cluster address is of CTA scope where it names none, and says nothing to the CTA
    that it is for."""
    csrc = os.path.join(os.path.dirname(moe.LIB_PATH), "csrc")
    found = []
    for name in os.listdir(csrc):
        found += re.findall(r'"(mbarrier\.arrive[^ ]*shared::cluster[^ ]*)', open(os.path.join(csrc, name)).read())
    assert len(found) >= 2 and all(".cluster.shared::cluster" in f for f in found), found


# ------------------------------------------------------------------ on the GPU

def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(g, rows, cols):
    return torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)


def scales(g, n, size=0.01):
    return (0.1 + torch.rand(n, generator=g, device="cuda")) * size


def least(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps


def check(y, x, xs, w, ws, swiglu=False, residual=None):
    """y of the rows x against one weight matrix w."""
    e = torch.finfo(y.dtype).eps / 2
    v = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    if swiglu:
        pairs = v.view(v.shape[0], -1, 2, 16)
        g, up = (pairs[:, :, i].reshape(v.shape[0], -1) for i in (0, 1))
        v = g / (1 + torch.exp(-g)) * up
        bound = ((14 + 6 * g.abs()) * U + (2.0 ** -21 if y.dtype != torch.float32 else 0)) * v.abs()
        bound = bound + (g * up).abs() * 2.0 ** -126
    else:
        r = residual.double() if residual is not None else torch.zeros_like(v)
        bound = 3 * U * v.abs() + U * (v.abs() + r.abs())
        v = v + r
    assert torch.all((y.double() - v).abs() <= bound + e * (v.abs() + bound) + least(y.dtype))


def dense(R, N, K, dtype, swiglu=False, residual=False, seed=1):
    g = gen(seed)
    cfg = q8.MatmulConfig(R, N, K, swiglu=swiglu, dtype=dtype)
    x, w = ints(g, R, K), ints(g, N, K)
    # scales that bring results to a few units
    xs, ws = scales(g, R), scales(g, N, 0.1 / K ** 0.5)
    res = torch.randn(R, cfg.columns, generator=g, device="cuda").to(dtype) if residual else None
    work = q8.workspace(cfg)
    y = q8.matmul(cfg, x, xs, w, ws, work, residual=res)
    check(y, x, xs, w, ws, swiglu, res)
    assert torch.equal(y, q8.matmul(cfg, x, xs, w, ws, work, residual=res))
    assert moe.device_error(work) == 0


# one row to several tiles of either kind, channels and K off every tile size, one k-block to many, split and not
SHAPES = [(1, 1, 16), (1, 128, 128), (1, 6144, 1536), (2, 100, 144), (31, 129, 256), (33, 4096, 528), (64, 6144, 12288),
          (65, 640, 384), (63, 24576, 2048), (127, 257, 4096), (129, 256, 128), (255, 1000, 2064), (256, 512, 1024),
          (257, 1001, 528), (300, 6144, 4112), (1000, 777, 1040), (2049, 2048, 512)]


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,K", SHAPES)
def test_dense(R, N, K):
    for i, dtype in enumerate(DT):
        dense(R, N, K, dtype, residual=(R + i) % 2 == 0, seed=i)


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,K", [(1, 32, 32), (3, 96, 400), (64, 24576, 1024), (100, 4096, 6144), (257, 4064, 272),
                                   (1111, 736, 2048)])
def test_dense_swiglu(R, N, K):
    for i, dtype in enumerate(DT):
        dense(R, N, K, dtype, swiglu=True, seed=i)


# 48 MB of token rows are 3 token blocks of a pair, 12 of a single CTA: a whole chunk of them and a part of one
@pytest.mark.gpu
@pytest.mark.parametrize("R,N", [(1100, 1100), (1100, 4300), (1100, 300), (1664, 4300)])
def test_long_rows_in_chunks_of_token_blocks(R, N):
    dense(R, N, 65536, torch.bfloat16, residual=True)


@pytest.mark.gpu
@pytest.mark.parametrize("G,rows", [(40, 1000), (3, 2500)])  # single CTAs, pairs
def test_one_group_in_chunks(G, rows):
    K, N = 65536, 300
    counts = [3] * G
    counts[G // 2] = rows
    g, R = gen(12), sum(counts)
    cfg = q8.MatmulConfig(R, N, K, groups=G, dtype=torch.float32)
    x, w, xs, ws = ints(g, R, K), ints(g, G * N, K), scales(g, R), scales(g, G * N, 0.1 / K ** 0.5)
    work, off = q8.workspace(cfg), offsets_of(counts)
    out = torch.full((R, N), 7.0, device="cuda")
    q8.matmul(cfg, x, xs, w, ws, work, offsets=off, out=out)
    edges = off.tolist()
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        check(out[a:b], x[a:b], xs[a:b], w[i * N:(i + 1) * N], ws[i * N:(i + 1) * N])
    assert moe.device_error(work) == 0


def offsets_of(counts):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.tensor(counts, device="cuda").cumsum(0)
    return off


GROUPS = [
    ([3, 0, 1, 64, 0, 65, 2], 0),            # few rows each: single CTAs, empty groups
    ([0, 0, 0], 5),                          # nothing at all, rows behind the last group
    ([700, 0, 130, 256, 1, 257, 512], 9),    # pairs: full and ragged tiles, one row
    ([0] * 100 + [33] + [0] * 100 + [1] * 56, 0),
    ([1000], 24),                            # one group that ends before the rows do
]


@pytest.mark.gpu
@pytest.mark.parametrize("counts,behind", GROUPS)
@pytest.mark.parametrize("N,K,swiglu", [(256, 384, False), (352, 528, True), (1000, 128, False)])
def test_groups(counts, behind, N, K, swiglu):
    G, R, dtype = len(counts), sum(counts) + behind, DT[(N + behind) % 3]
    g = gen(5)
    cfg = q8.MatmulConfig(R, N, K, groups=G, swiglu=swiglu, dtype=dtype)
    x, w = ints(g, R, K), ints(g, G * N, K)
    xs, ws = scales(g, R), scales(g, G * N, 0.1 / K ** 0.5)
    work, off = q8.workspace(cfg), offsets_of(counts)
    res = None if swiglu else torch.randn(R, N, generator=g, device="cuda").to(dtype)
    out = torch.full((R, cfg.columns), 7.0, device="cuda").to(dtype)
    q8.matmul(cfg, x, xs, w, ws, work, offsets=off, residual=res, out=out)
    edges = off.tolist()
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        if b > a:
            check(out[a:b], x[a:b], xs[a:b], w[i * N:(i + 1) * N], ws[i * N:(i + 1) * N], swiglu,
                  None if res is None else res[a:b])
    assert bool((out[edges[-1]:] == 7).all()) and moe.device_error(work) == 0


@pytest.mark.gpu
def test_bad_offsets_are_flagged():
    G, R, N, K = 4, 200, 64, 64
    g = gen(6)
    cfg = q8.MatmulConfig(R, N, K, groups=G)
    x, w, xs, ws = ints(g, R, K), ints(g, G * N, K), scales(g, R), scales(g, G * N)
    work = q8.workspace(cfg)
    good = offsets_of([50, 50, 50, 50])
    want = q8.matmul(cfg, x, xs, w, ws, work, offsets=good)
    for bad in ([0, 50, 40, 150, 200], [0, 50, 100, 150, 201], [0, -1, 100, 150, 200], [1, 50, 100, 150, 200],
                [0, 200, 0, 200, 0], [0, 200, 2 ** 31 - 1, 150, 200]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        q8.matmul(cfg, x, xs, w, ws, work, offsets=off)
        assert moe.device_error(work) == 5, bad
    off = torch.tensor([0, 50, 40, 150, 200], dtype=torch.int32, device="cuda")
    y = torch.zeros_like(want)
    q8.matmul(cfg, x, xs, w, ws, work, offsets=off, out=y)
    assert torch.equal(y[150:], want[150:])  # a valid group keeps its rows beside a rejected one
    assert moe.device_error(work) == 5


@pytest.mark.gpu
@pytest.mark.parametrize("R", [40, 300])
def test_extreme_values(R):
    N, K = 96, 65536
    x = torch.full((R, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    x[3] = 0
    one = torch.ones
    cfg = q8.MatmulConfig(R, N, K, dtype=torch.float32)
    work = q8.workspace(cfg)
    xs = one(R, device="cuda")
    xs[5] = float("nan")
    y = q8.matmul(cfg, x, xs, w, one(N, device="cuda"), work)
    want = torch.tensor([2.0 ** 30, -128.0 * 127 * K], device="cuda").repeat(N // 2)
    assert torch.equal(y[0], want) and torch.equal(y[R - 1], want) and not y[3].any() and torch.isnan(y[5]).all()
    half = q8.MatmulConfig(R, N, K, dtype=torch.float16)
    y = q8.matmul(half, x, xs, w, one(N, device="cuda"), work)
    assert y[0, 0].item() == 65504 and y[0, 1].item() == -65504 and torch.isnan(y[5]).all()
    assert moe.device_error(work) == 8 and moe.device_error(work) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,dtype", [(50, 200, torch.bfloat16), (300, 100, torch.float16), (70, 131, torch.float32)])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1)])
def test_strides_and_in_place(R, N, dtype, pad, shift):
    K, g = 160, gen(7)
    x = ints(g, R, K + 48)[:, 16:16 + K]
    w, xs, ws = ints(g, N, K), scales(g, R), scales(g, N)
    cfg = q8.MatmulConfig(R, N, K, dtype=dtype)
    work = q8.workspace(cfg)
    buf = torch.randn(R, N + pad, generator=g, device="cuda").to(dtype)
    res = buf[:, shift:shift + N]
    was = buf.clone()
    q8.matmul(cfg, x, xs, w, ws, work, residual=res, out=res)
    check(res, x, xs, w, ws, residual=was[:, shift:shift + N])
    assert torch.equal(buf[:, :shift], was[:, :shift]) and torch.equal(buf[:, shift + N:], was[:, shift + N:])


@pytest.mark.gpu
def test_streams_graphs_and_shared_workspaces():
    """Two captured products of the same workspace, replayed in turn on one stream; and an empty product."""
    g = gen(8)
    small, large = q8.MatmulConfig(8, 512, 4096), q8.MatmulConfig(300, 512, 4096)
    work = q8.workspace(small, large)
    w, ws = ints(g, 512, 4096), scales(g, 512)
    xa, xb, sa, sb = ints(g, 8, 4096), ints(g, 300, 4096), scales(g, 8), scales(g, 300)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ya = q8.matmul(small, xa, sa, w, ws, work, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check(ya, xa, sa, w, ws)
    graphs = []
    yb = torch.empty(300, 512, dtype=torch.bfloat16, device="cuda")
    for cfg, x, sc, y in ((small, xa, sa, ya), (large, xb, sb, yb)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q8.matmul(cfg, x, sc, w, ws, work, out=y)
        graphs.append(graph)
    for _ in range(3):
        xa.add_(1)
        xb.add_(1)
        for graph in graphs:
            graph.replay()
        check(ya, xa, sa, w, ws)
        check(yb, xb, sb, w, ws)
    y = q8.matmul(q8.MatmulConfig(0, 512, 4096), xa[:0], sa[:0], w, ws, work)
    assert y.shape == (0, 512) and moe.device_error(work) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("R", [16, 600])
def test_timeout_is_reported_and_context_survives(R, monkeypatch):
    g = gen(9)
    cfg = q8.MatmulConfig(R, 512, 512)
    x, w, xs, ws, work = ints(g, R, 512), ints(g, 512, 512), scales(g, R), scales(g, 512), q8.workspace(cfg)
    monkeypatch.setenv("SRM_MOE_INJECT_STALL", "1")
    q8.matmul(cfg, x, xs, w, ws, work)
    assert moe.device_error(work) == 6
    monkeypatch.delenv("SRM_MOE_INJECT_STALL")
    for _ in range(2):
        check(q8.matmul(cfg, x, xs, w, ws, work), x, xs, w, ws)
    q8.init_workspace(work)
    check(q8.matmul(cfg, x, xs, w, ws, work), x, xs, w, ws)
    assert moe.device_error(work) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("R,N,K", [(5, 700, 2048), (64, 24576, 1024), (300, 1000, 4096), (3000, 4096, 256)])
def test_workspace_without_its_control_words(R, N, K):
    """Only the first 256 bytes zero, the rest anything: whole tiles in a fixed stride, the same results."""
    g = gen(11)
    cfg = q8.MatmulConfig(R, N, K)
    x, w, xs, ws = ints(g, R, K), ints(g, N, K), scales(g, R), scales(g, N)
    good = q8.matmul(cfg, x, xs, w, ws, q8.workspace(cfg))
    work = torch.randint(0, 256, (q8.workspace_bytes(cfg),), generator=g, device="cuda", dtype=torch.uint8)
    work[:256] = 0
    for _ in range(2):
        assert torch.equal(q8.matmul(cfg, x, xs, w, ws, work), good)
    q8.init_workspace(work)
    for _ in range(3):  # the counters are back at zero after each call
        assert torch.equal(q8.matmul(cfg, x, xs, w, ws, work), good)
    assert moe.device_error(work) == 0


@pytest.mark.gpu
def test_binding_refusals():
    g = gen(10)
    cfg = q8.MatmulConfig(4, 64, 64, groups=2)
    x, w, xs, ws, work = ints(g, 4, 64), ints(g, 128, 64), scales(g, 4), scales(g, 128), q8.workspace(cfg)
    off = offsets_of([2, 2])
    with pytest.raises(moe.MoeError):
        q8.matmul(cfg, x, xs, w, ws, work)  # groups without offsets
    with pytest.raises(ValueError):
        q8.matmul(cfg, x, xs, w, ws, work, offsets=off[:2])
    with pytest.raises(TypeError):
        q8.matmul(cfg, x, xs, w, ws, work, offsets=off.long())
    with pytest.raises(ValueError):
        q8.matmul(cfg, x, xs, w[:64], ws, work, offsets=off)
    with pytest.raises(moe.MoeError):
        q8.matmul(cfg, ints(g, 4, 72)[:, 8:], xs, w, ws, work, offsets=off)  # rows off 16 bytes
    with pytest.raises(moe.MoeError):
        q8.workspace(q8.MatmulConfig(4, 64, 65))
    assert moe.device_error(work) == 0
