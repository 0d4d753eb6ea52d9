"""Rows sorted by expert and back (include/srm_rows.h) and their gradients against the definition in 64 bits and
against differences, and the refusals.

Tolerances.  u = 2^-24 is fp32's half step, e_t half a step of the result's type.  A sum of n products in fp32, each
fused with its addition, is off by at most n u sum |terms|; one more for the residual, then one rounding to the type.
A gradient of a weight is a dot product over H: a lane's chain of fused products, five shuffles and at most eight
partial sums, H / 32 + 13 at most: (H / 32 + 13) u sum |terms|."""
import ctypes
import os
import subprocess

import pytest
import torch

from sigmoid_routed_mixture_b200 import moe, q8, rows

U = 2.0 ** -24
DT = [torch.bfloat16, torch.float16, torch.float32]
A = ctypes.c_void_p(0x100000)  # aligned; never dereferenced, validation fails first
ODD = ctypes.c_void_p(0x100001)


# ------------------------------------------------------------------ refusals (CPU)

def c_cfg(T=4, H=64, E=8, K=2, shared=1, dtype=0, slot=1, ld=None):
    ld = H if ld is None else ld
    return rows._Cfg(T, H, E, K, shared, dtype, slot, ld, ld, ld, ld)


def calls(c):
    L, r = rows.lib(), ctypes.byref(c)
    return [L.moe_rows_sort(r, A, None, A, A, A, A, None, A, None), L.moe_rows_unsort(r, A, A, A, A, A, A, None),
            L.moe_rows_sort_grad(r, A, A, A, A, None), L.moe_rows_unsort_grad(r, A, A, A, A, A, A, A, None)]


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(K=0), 1), (dict(K=9), 1), (dict(E=0), 1), (dict(shared=2), 1),
    (dict(dtype=5), 1), (dict(ld=63), 1), (dict(ld=(1 << 31) + 1), 1), (dict(E=257), 2), (dict(K=17, E=20), 2),
    (dict(H=(1 << 20) + 1), 2), (dict(T=1 << 30), 2),
])
def test_shapes_refused(kw, code):
    assert calls(c_cfg(**kw)) == [code] * 4


def test_types_and_pointers_refused():
    L = rows.lib()
    c = ctypes.byref(c_cfg())
    int8 = ctypes.byref(c_cfg(dtype=3))
    assert L.moe_rows_unsort(int8, A, A, A, A, A, A, None) == 1
    assert L.moe_rows_sort_grad(int8, A, A, A, A, None) == 1
    assert L.moe_rows_unsort_grad(int8, A, A, A, A, A, A, A, None) == 1
    assert L.moe_rows_unsort(ctypes.byref(c_cfg(slot=3)), A, A, A, A, A, A, None) == 1
    assert L.moe_rows_sort(c, None, None, A, A, A, A, None, A, None) == 1
    assert L.moe_rows_sort(c, A, A, A, A, A, A, None, A, None) == 1  # scales in, none out
    assert L.moe_rows_sort(c, A, None, A, A, A, A, None, None, None) == 1
    assert L.moe_rows_sort(c, ODD, None, A, A, A, A, None, A, None) == 3
    assert L.moe_rows_sort(c, A, None, A, A, A, A, None, ctypes.c_void_p(0x100080), None) == 3
    assert L.moe_rows_unsort(c, A, A, None, A, A, A, None) == 1
    assert L.moe_rows_unsort(c, A, ODD, A, A, A, A, None) == 3
    assert L.moe_rows_sort_grad(None, A, A, A, A, None) == 1
    assert L.moe_rows_sort_grad(c, A, A, ODD, A, None) == 3
    assert L.moe_rows_unsort_grad(c, A, A, A, A, None, None, A, None) == 1
    assert L.moe_rows_unsort_grad(c, A, None, A, A, A, A, A, None) == 1
    assert L.moe_rows_unsort_grad(c, A, A, A, A, ODD, A, A, None) == 3
    apart = c_cfg()
    apart.ld_residual = apart.ld_dys = 72  # in place, their rows elsewhere
    assert L.moe_rows_unsort(ctypes.byref(apart), A, A, A, A, A, A, None) == 1
    assert L.moe_rows_unsort_grad(ctypes.byref(apart), A, A, A, A, A, A, A, None) == 1
    empty = ctypes.byref(c_cfg(T=0))
    assert L.moe_rows_sort(empty, *[None] * 9) == 0 and L.moe_rows_unsort(empty, *[None] * 7) == 0
    assert L.moe_rows_sort_grad(empty, *[None] * 5) == 0 and L.moe_rows_unsort_grad(empty, *[None] * 8) == 0


def test_binding_refuses_host_tensors():
    cfg = rows.Config(4, 8, 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        rows.sort(cfg, torch.zeros(4, 8, dtype=torch.bfloat16), None, None, None)


def test_walk_of_the_inverse_stays_in_range(tmp_path):
    """rows_invert_kernel's indices over the last two steps of the grid, up to as many positions as are accepted
    (2^31 - 1): each once and none outside."""
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text("""#include <cstdlib>
#include <initializer_list>
#include "grid_walk.h"
int main() {
  const int64_t step = 8 * 148 * 256;
  for (int64_t n : {(int64_t(1) << 31) - 1, (int64_t(1) << 31) - step, int64_t(2147400000), int64_t(1000003)}) {
    const int64_t start = (n / step > 1 ? n / step - 1 : 0) * step;
    int64_t seen = 0, sum = 0;
    for (int64_t first = 0; first < step; ++first) {
      srm::grid_walk(start + first, step, n, [&](int i) {
        if (i < start || i >= n) std::exit(2);
        ++seen;
        sum += i - start;
      });
    }
    const int64_t m = n - start;
    if (seen != m || sum != m * (m - 1) / 2) return 1;
  }
  return 0;
}
""")
    csrc = os.path.join(os.path.dirname(moe.LIB_PATH), "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


def test_overlapped_kernels_promise_nothing_about_their_inputs():
    """A kernel that starts before the one ahead of it has ended may not call its inputs constant for its lifetime:
    files that launch this way have no __restrict__ pointers and no loads by the read-only path."""
    csrc = os.path.join(os.path.dirname(moe.LIB_PATH), "csrc")
    texts = {n: open(os.path.join(csrc, n)).read() for n in os.listdir(csrc)}
    files = [n for n in texts if "previous_done()" in texts[n] and n != "launch.cuh"]
    assert len(files) >= 3
    for n in files:
        code = "\n".join(line.split("//")[0] for line in texts[n].splitlines())
        for word in ("__restrict__", "__ldg", "global.nc"):
            assert word not in code, (n, word)


# ------------------------------------------------------------------ on the GPU

def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def routing(T, E, K, shared, seed, idx=None):
    """(gate, offsets, sorted, pos) with moe.permute's order, made here from its definition."""
    g = gen(seed)
    if idx is None:
        idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K]
    gate = torch.randn(T, K, generator=g, device="cuda")
    flat = idx.reshape(-1)
    ids = flat.argsort(stable=True)
    counts = torch.bincount(flat, minlength=E)
    if shared:
        ids = torch.cat([ids, torch.arange(T * K, T * K + T, device="cuda")])
    counts = torch.cat([counts, torch.tensor([T if shared else 0], device="cuda")])
    offsets = torch.zeros(E + 2, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    pos = torch.empty(ids.numel(), dtype=torch.int32, device="cuda")
    pos[ids] = torch.arange(ids.numel(), dtype=torch.int32, device="cuda")
    return gate, offsets, ids.to(torch.int32), pos


def token_of(ids, T, K):
    return torch.where(ids < T * K, ids // max(K, 1), ids - T * K).long()


def half(t):
    return torch.finfo(t).eps / 2


def least(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps


def check_unsort(y, ys, gate, pos, cfg, residual=None):
    T, K = cfg.T, cfg.K
    p = pos.long()
    picked = torch.where(p[:, None] >= 0, ys.double()[p.clamp(min=0)], 0.0)
    terms = picked[: T * K].view(T, K, -1) * (gate.double()[..., None] if gate is not None else 1.0)
    if cfg.has_shared:
        terms = torch.cat([terms, picked[T * K:].view(T, 1, -1)], 1)
    exact, size = terms.sum(1), terms.abs().sum(1)
    if residual is not None:
        exact, size = exact + residual.double(), size + residual.double().abs()
    bound = (K + 2) * U * size
    assert torch.all((y.double() - exact).abs() <= bound + half(y.dtype) * (exact.abs() + bound) + least(y.dtype))


def check_grad(dys, dgate, dy, ys, gate, pos, cfg, before):
    T, K, H = cfg.T, cfg.K, cfg.H
    p = pos.long()
    w = torch.ones(cfg.rows, dtype=torch.float64, device="cuda")
    if gate is not None:
        w[: T * K] = gate.double().reshape(-1)
    tok = token_of(torch.arange(cfg.rows, device="cuda"), T, K)
    held = p >= 0
    want = w[held, None] * dy.double()[tok[held]]
    got = dys[p[held]].double()
    assert torch.all((got - want).abs() <= (half(dys.dtype) + 2 * U) * want.abs() + least(dys.dtype))
    rest = torch.ones(cfg.rows, dtype=torch.bool, device="cuda")
    rest[p[held]] = False
    assert torch.equal(dys[rest], before[rest])  # rows that no assignment holds are left as they were
    rr = torch.where(held[: T * K, None], ys.double()[p[: T * K].clamp(min=0)], 0.0).view(T, K, H)
    terms = rr * dy.double()[:, None]
    assert torch.all((dgate.double() - terms.sum(2)).abs() <= (H / 32 + 13) * U * terms.abs().sum(2) + 2.0 ** -149)


SHAPES = [(1, 1, 1, 1, True), (1, 6144, 256, 8, True), (3, 17, 5, 5, False), (64, 2048, 64, 4, True),
          (129, 264, 16, 16, True), (300, 1541, 256, 8, True), (5, 40008, 4, 2, True), (5000, 64, 8, 3, False),
          (700, 4104, 32, 9, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H,E,K,shared", SHAPES)
def test_there_and_back(T, H, E, K, shared, dtype):
    slot = DT[(DT.index(dtype) + T) % 3]
    cfg = rows.Config(T, H, E, K, shared, dtype, slot)
    gate, offsets, ids, pos = routing(T, E, K, shared, 1)
    g, ws = gen(2), rows.workspace()
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    xs, got_pos = rows.sort(cfg, x, offsets, ids, ws)
    assert torch.equal(xs, x[token_of(ids, T, K)]) and torch.equal(got_pos, pos)
    ys = torch.randn(cfg.rows, H, generator=g, device="cuda").to(slot)
    residual = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    for gt, res in ((gate, None), (None, residual), (gate, residual)):
        y = rows.unsort(cfg, ys, gt, pos, ws, residual=res)
        check_unsort(y, ys, gt, pos, cfg, res)
        assert torch.equal(y, rows.unsort(cfg, ys, gt, pos, ws, residual=res))
    dy = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    for gt in (gate, None):
        before = torch.full_like(ys, 7)
        dys, dgate = rows.unsort_grad(cfg, dy, ys, gt, pos, ws, out=before.clone())
        check_grad(dys, dgate, dy, ys, gt, pos, cfg, before)
        again, dgate2 = rows.unsort_grad(cfg, dy, ys, gt, pos, ws)
        assert torch.equal(again, dys) and torch.equal(dgate2, dgate)
        kept = ys.clone()
        in_place, dgate2 = rows.unsort_grad(cfg, dy, kept, gt, pos, ws, out=kept)
        assert torch.equal(in_place, dys) and torch.equal(dgate2, dgate)
    dxs = torch.randn(cfg.rows, H, generator=g, device="cuda").to(dtype)
    dx = rows.sort_grad(cfg, dxs, pos, ws)
    check_unsort(dx, dxs, None, pos, rows.Config(T, H, E, K, shared, dtype, dtype))
    assert moe.device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("H,ld", [(64, 64), (64, 80), (48, 49), (37, 40), (6144, 6160)])
def test_int8_rows_with_scales(H, ld):
    T, E, K = 77, 9, 3
    cfg = rows.Config(T, H, E, K, True, torch.int8)
    _, offsets, ids, pos = routing(T, E, K, True, 3)
    g, ws = gen(4), rows.workspace()
    x = torch.randint(-127, 128, (T, ld), generator=g, device="cuda", dtype=torch.int8)[:, :H]
    scale = torch.rand(T, generator=g, device="cuda")
    out = torch.full((cfg.rows, ld + 1), 5, dtype=torch.int8, device="cuda")
    xs, xs_scale, got = rows.sort(cfg, x, offsets, ids, ws, x_scale=scale, out=out[:, :H])
    tok = token_of(ids, T, K)
    assert torch.equal(xs, x[tok]) and torch.equal(xs_scale, scale[tok]) and torch.equal(got, pos)
    assert bool((out[:, H:] == 5).all())


@pytest.mark.gpu
@pytest.mark.parametrize("ld,offset", [(64, 0), (72, 0), (67, 0), (72, 3)])
def test_strides(ld, offset):
    T, H, E, K = 41, 64, 6, 2
    cfg = rows.Config(T, H, E, K, True, torch.bfloat16, torch.float16)
    gate, offsets, ids, pos = routing(T, E, K, True, 5)
    g, ws = gen(6), rows.workspace()

    def view(n, dtype):
        return torch.randn(n * ld + offset, generator=g, device="cuda").to(dtype).as_strided((n, H), (ld, 1), offset)

    x, ys, res, dy = view(T, cfg.dtype), view(cfg.rows, cfg.slot_dtype), view(T, cfg.dtype), view(T, cfg.dtype)
    xs, _ = rows.sort(cfg, x, offsets, ids, ws, out=view(cfg.rows, cfg.dtype))
    assert torch.equal(xs, x[token_of(ids, T, K)])
    check_unsort(rows.unsort(cfg, ys, gate, pos, ws, residual=res), ys, gate, pos, cfg, res)
    was = res.clone()
    rows.unsort(cfg, ys, gate, pos, ws, residual=res, out=res)
    check_unsort(res, ys, gate, pos, cfg, was)
    before = view(cfg.rows, cfg.slot_dtype)
    dys, dgate = rows.unsort_grad(cfg, dy, ys, gate, pos, ws, out=before)
    check_grad(dys, dgate, dy, ys, gate, pos, cfg, before)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H,ld,offset", [(41, 64, 72, 0), (41, 64, 67, 3), (1200, 37, 40, 1), (5, 4099, 4104, 8)])
def test_nothing_beside_the_rows_is_written(T, H, ld, offset, dtype):
    """Strided results inside larger buffers, and positions that no row holds: all else stays as it was."""
    E, K = 6, 2
    cfg = rows.Config(T, H, E, K, True, dtype, dtype)
    gate, offsets, ids, pos = routing(T, E, K, True, 17)
    offsets, pos = offsets.clone(), pos.clone()
    offsets[E + 1] -= 2  # the last two positions hold no row
    pos[ids[-2:].long()] = -1
    g, ws = gen(18), rows.workspace()

    def buffer(n):
        flat = torch.randn(n * ld + offset + 5, generator=g, device="cuda").to(dtype)
        return flat, flat.as_strided((n, H), (ld, 1), offset)

    def others(flat, n):
        """All of a buffer but the view's first n rows."""
        keep = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
        keep.as_strided((n, H), (ld, 1), offset).fill_(False)
        return flat[keep]

    x, ys, dy = buffer(T)[1], buffer(cfg.rows)[1], buffer(T)[1]
    held = cfg.rows - 2
    for n, call in ((held, lambda out: rows.sort(cfg, x, offsets, ids, ws, out=out)),
                    (T, lambda out: rows.unsort(cfg, ys, gate, pos, ws, out=out)),
                    (T, lambda out: rows.sort_grad(cfg, ys, pos, ws, out=out)),
                    (held, lambda out: rows.unsort_grad(cfg, dy, ys, gate, pos, ws, out=out))):
        flat, view = buffer(T if n == T else cfg.rows)
        before = flat.clone()
        call(view)
        assert torch.equal(others(flat, n), others(before, n))
        plain = call(torch.zeros(view.shape, dtype=dtype, device="cuda"))
        plain = plain[0] if isinstance(plain, tuple) else plain
        assert torch.equal(view[:n], plain[:n])
    assert moe.device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [300, 900])  # the inverse in one launch, and in several
def test_after_permute_with_ids_out_of_range(T):
    """moe_permute skips and flags an id out of range: its assignment has no row, and adds nothing."""
    H, E, K = 256, 16, 4
    block = moe.Config(T=T, H=H, I=128, E=E, K=K)
    cfg = rows.Config.of(block)
    assert (cfg.rows <= 4096) == (T == 300)
    idx = torch.rand(T, E, generator=gen(7), device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
    idx[3, 1], idx[200, 0], idx[299] = -1, E, 1000
    ws = moe.workspace(block)
    _, offsets, ids = moe.permute(block, idx, ws)
    assert moe.device_error(ws) == 5
    gone = [3 * K + 1, 200 * K] + list(range(299 * K, 300 * K))
    n = cfg.rows - len(gone)
    ids[n:] = 123456789  # not written by the permutation, and not to be read
    x = torch.randn(T, H, generator=gen(8), device="cuda").to(torch.bfloat16)
    out = torch.full((cfg.rows, H), 3.0, dtype=torch.bfloat16, device="cuda")
    xs, pos = rows.sort(cfg, x, offsets, ids, ws, out=out)
    assert torch.nonzero(pos < 0).flatten().tolist() == gone and moe.device_error(ws) == 0
    assert torch.equal(xs[:n], x[token_of(ids[:n], T, K)]) and bool((xs[n:] == 3).all())
    gate = torch.randn(T, K, generator=gen(9), device="cuda")
    ys = torch.randn(cfg.rows, H, generator=gen(10), device="cuda").to(torch.float16)
    ys[n:] = float("nan")  # rows behind the last one
    y = rows.unsort(cfg, ys, gate, pos, ws)
    check_unsort(y, torch.nan_to_num(ys), gate, pos, cfg)
    before = torch.full_like(ys, 7)
    dys, dgate = rows.unsort_grad(cfg, x, ys, gate, pos, ws, out=before.clone())
    check_grad(dys, dgate, x, torch.nan_to_num(ys), gate, pos, cfg, before)
    assert not dgate.reshape(-1)[gone].any() and moe.device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 2000])  # the inverse in one launch, and in several
def test_bad_ids_and_positions_are_flagged(T):
    H, E, K = 32, 4, 2
    cfg = rows.Config(T, H, E, K)
    gate, offsets, ids, pos = routing(T, E, K, True, 11)
    x = torch.randn(T, H, generator=gen(12), device="cuda").to(torch.bfloat16)
    ws = rows.workspace()
    bad = ids.clone()
    bad[[4, 9]] = torch.tensor([-7, cfg.rows], dtype=torch.int32, device="cuda")
    xs, p = rows.sort(cfg, x, offsets, bad, ws)
    assert moe.device_error(ws) == 5 and moe.device_error(ws) == 0
    assert sorted(torch.nonzero(p < 0).flatten().tolist()) == sorted(ids[[4, 9]].tolist())
    for total in (-1, cfg.rows + 1):
        wrong = offsets.clone()
        wrong[E + 1] = total
        _, p = rows.sort(cfg, x, wrong, ids, ws)
        assert bool((p == -1).all()) and moe.device_error(ws) == 5
    ys = torch.randn(cfg.rows, H, generator=gen(13), device="cuda").to(torch.float16)
    wrong = pos.clone()
    wrong[[0, 7]] = torch.tensor([cfg.rows, -2], dtype=torch.int32, device="cuda")
    as_gone = pos.clone()
    as_gone[[0, 7]] = -1
    assert torch.equal(rows.unsort(cfg, ys, gate, wrong, ws), rows.unsort(cfg, ys, gate, as_gone, ws))
    assert moe.device_error(ws) == 5
    dy = x.clone()
    a = rows.unsort_grad(cfg, dy, ys, gate, wrong, ws, out=torch.zeros_like(ys))
    assert moe.device_error(ws) == 5
    b = rows.unsort_grad(cfg, dy, ys, gate, as_gone, ws, out=torch.zeros_like(ys))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and moe.device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 2000])  # the inverse in one launch, and in several
def test_id_in_two_positions(T):
    """The later position takes the row, in every run; the other's row of xs stays as it was."""
    H, E, K = 32, 4, 2
    cfg = rows.Config(T, H, E, K)
    gate, offsets, ids, pos = routing(T, E, K, True, 14)
    x = torch.randn(T, H, generator=gen(15), device="cuda").to(torch.bfloat16)
    twice = ids.clone()
    P = cfg.rows
    twice[1::3] = ids[0:P - 1:3][:len(twice[1::3])]  # each third id in the next position too
    last = torch.full((P,), -1, dtype=torch.int64, device="cuda")
    last.scatter_reduce_(0, twice.long(), torch.arange(P, device="cuda"), "amax")
    ws = rows.workspace()
    for _ in range(3):
        out = torch.full((P, H), 3.0, dtype=torch.bfloat16, device="cuda")
        xs, p = rows.sort(cfg, x, offsets, twice, ws, out=out)
        assert torch.equal(p.long(), last) and moe.device_error(ws) == 5
        want = torch.full_like(out, 3.0)
        held = last[last >= 0]
        want[held] = x[token_of(twice, T, K)][held]
        assert torch.equal(xs, want)


@pytest.mark.gpu
def test_gradients_against_differences():
    """A scalar of the whole way (sort, a linear map per position, unsort) in fp32 rows, differenced."""
    T, H, E, K = 6, 16, 5, 2
    cfg = rows.Config(T, H, E, K, True, torch.float32, torch.float32)
    gate, offsets, ids, pos = routing(T, E, K, True, 14)
    g, ws = gen(15), rows.workspace()
    x = torch.randn(T, H, generator=g, device="cuda")
    m = torch.randn(cfg.rows, H, generator=g, device="cuda")
    r = torch.randn(T, H, generator=g, device="cuda")

    def loss(x_, gate_):
        xs, p = rows.sort(cfg, x_.float(), offsets, ids, ws)
        return (rows.unsort(cfg, xs * m, gate_.float(), p, ws).double() * r.double()).sum()

    xs, p = rows.sort(cfg, x, offsets, ids, ws)
    dys, dgate = rows.unsort_grad(cfg, r, xs * m, gate, p, ws)
    dx = rows.sort_grad(cfg, dys * m, p, ws)
    h = 2.0 ** -6  # the loss is linear in each single entry, so the step only has to beat fp32's rounding
    for t_, d in ((0, dx), (1, dgate)):
        for i in range(0, d.numel(), 3):
            plus, minus = [x.clone(), gate.clone()], [x.clone(), gate.clone()]
            plus[t_].view(-1)[i] += h
            minus[t_].view(-1)[i] -= h
            slope = (loss(*plus) - loss(*minus)) / (2 * h)
            # y's entries are below 64, off by (K + 2) u 64 each; H of them enter, each weighted below 4
            assert abs(slope.item() - d.view(-1)[i].item()) <= H * 4 * (K + 2) * U * 64 / h + 1e-5 * abs(slope.item())


@pytest.mark.gpu
def test_capture_other_stream_and_dense_group():
    T, H = 50, 128
    cfg = rows.Config(T, H, 0, 0, True, torch.bfloat16, torch.bfloat16)  # one group: the dense form
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ids = torch.arange(T, dtype=torch.int32, device="cuda")
    x, ws = torch.randn(T, H, device="cuda").to(torch.bfloat16), rows.workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    xs, pos = rows.sort(cfg, x, offsets, ids, ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(xs, x) and torch.equal(pos, ids)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows.sort(cfg, x, offsets, ids, ws, out=xs, pos=pos)
        y = rows.unsort(cfg, xs, None, pos, ws)
    x.add_(1)
    graph.replay()
    assert torch.equal(y, x)
    assert moe.device_error(ws) == 0


@pytest.mark.gpu
def test_binding_refusals():
    T, H, E, K = 4, 8, 4, 2
    cfg = rows.Config(T, H, E, K)
    gate, offsets, ids, pos = routing(T, E, K, True, 16)
    x, ws = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), rows.workspace()
    ys = torch.zeros(cfg.rows, H, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        rows.sort(cfg, x[:2], offsets, ids, ws)
    with pytest.raises(TypeError):
        rows.sort(cfg, x.half(), offsets, ids, ws)
    with pytest.raises(ValueError):
        rows.sort(cfg, x, offsets[:-1], ids, ws)
    with pytest.raises(ValueError):
        rows.sort(cfg, x, offsets, ids, ws, xs_scale=gate[:, 0])
    with pytest.raises(TypeError):
        rows.unsort(cfg, ys, gate.half(), pos, ws)
    with pytest.raises(TypeError):
        rows.unsort(cfg, ys, gate, pos, ws[:10])
    with pytest.raises(moe.MoeError):
        rows.sort(rows.Config(T, H, E, 5), x, offsets, torch.zeros(T * 6, dtype=torch.int32, device="cuda"), ws)
    assert q8.DTYPES[torch.int8] == 3
