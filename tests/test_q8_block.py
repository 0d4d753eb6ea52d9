"""The 8-bit blocks (q8.MoeBlock, q8.DenseMlp): the row calls and products together, as they are used.

Two checks.  Bit for bit against the same public calls made one by one on fresh buffers.  And against the unquantised
formula in 64 bits, within what the roundings can do.  A rounding to 8 bits is off by an amount that is spread evenly
over its step s (variance s^2 / 12) and independent from element to element, so to first order an output's error is a
sum of independent terms whose variance follows from the formula's derivatives:
    from x:        sum_i J_i^2 sx^2 / 12,   J = W2 (diag(silu'(g) up) W1 + diag(silu(g)) W3) summed over the experts
    from W1, W3:   sum_j w2_j^2 |x|^2 ((silu'(g) up)_j^2 s1_j^2 + silu(g)_j^2 s3_j^2) / 12
    from h, W2:    sum_j w2_j^2 (sh^2 + (2^-10 h_j)^2) / 12 + |h|^2 s2^2 / 12          (fp16, then 8 bits)
Sums of evenly spread terms have thinner tails than a normal variable of their variance, for which eight standard
deviations leave 10^-15; a quarter is added for the second order.  The result's own rounding is 2^-9 relative (bf16)."""
import pytest
import torch

from sigmoid_routed_mixture_b200 import moe, q8, rows

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def step(v):
    """The step of a row's 8-bit form."""
    return v.abs().amax(-1) / 127


def mlp(x, w1, w3, w2):
    """The SwiGLU MLP of rows x in 64 bits; the derivative J [R, out, in] by x, and the variance of the
    error that the 8-bit weights and hidden rows bring."""
    g, up = x @ w1.t(), x @ w3.t()
    sig = torch.sigmoid(g)
    silu, slope = g * sig, sig * (1 + g * (1 - sig))
    h = silu * up
    a, b = slope * up, silu
    J = torch.matmul(w2 * a[:, None], w1) + torch.matmul(w2 * b[:, None], w3)
    x2, sh = (x * x).sum(1, keepdim=True), step(h)[:, None]
    per_h = x2 * (a * a * step(w1) ** 2 + b * b * step(w3) ** 2) + sh ** 2 + (h * 2.0 ** -10) ** 2
    var = (per_h @ (w2 * w2).t() + (h * h).sum(1, keepdim=True) * step(w2) ** 2) / 12
    return h @ w2.t(), J, var


def check(y, exact, J, var, sx):
    sigma = torch.sqrt(var + (J * J).sum(2) * sx[:, None] ** 2 / 12)
    bound = 10 * sigma
    assert torch.all((y.double() - exact).abs() <= bound + (exact.abs() + bound) * 2.0 ** -9)
    return sigma


def block(T, E, K, H, I, shared, seed, scale=2.5):
    cfg = moe.Config(T=T, H=H, I=I, E=E, K=K, routed_scale=scale, has_shared=shared)
    g = gen(seed)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").mul_(s[-1] ** -0.5).to(torch.bfloat16)  # noqa: E731
    w = dict(w1=draw(E, I, H), w3=draw(E, I, H), w2=draw(E, H, I))
    if shared:
        w.update(ws1=draw(I, H), ws3=draw(I, H), ws2=draw(H, I))
    router = torch.randn(E, H, generator=g, device="cuda") * 0.05
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    return cfg, q8.MoeBlock(cfg, router, bias, **w), w, g


def by_hand(blk, x, residual):
    """MoeBlock's steps on buffers of their own."""
    cfg, ws = blk.cfg, moe.workspace(blk.cfg)
    q, s = q8.quantize(x)
    idx, gate, _ = moe.route_packed(cfg, x, blk.router_packed, blk.bias, ws)
    _, offsets, ids = moe.permute(cfg, idx, ws)
    xs, xss, pos = rows.sort(rows.Config.of(cfg, dtype=torch.int8), q, offsets, ids, ws, x_scale=s)
    w13, s13, w2, s2 = blk.weights
    h = q8.matmul(blk.up, xs, xss, w13, s13, q8.workspace(blk.up), offsets=offsets)
    hq, hs = q8.quantize(h)
    ys = q8.matmul(blk.down, hq, hs, w2, s2, q8.workspace(blk.down), offsets=offsets)
    return rows.unsort(rows.Config.of(cfg), ys, gate, pos, ws, residual=residual), idx, gate


SHAPES = [(1, 4, 2, 256, 128, True), (64, 16, 4, 256, 128, True), (301, 8, 2, 512, 384, False),
          (1500, 4, 3, 256, 256, True), (17, 256, 16, 256, 128, True)]


@pytest.mark.parametrize("T,E,K,H,I,shared", SHAPES)
def test_moe_block(T, E, K, H, I, shared):
    cfg, blk, w, g = block(T, E, K, H, I, shared, 1)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    y = blk(x).clone()
    want, idx, gate = by_hand(blk, x, None)
    assert torch.equal(y, want) and blk.device_error() == 0
    xd = x.double()
    exact, var = torch.zeros_like(xd), torch.zeros_like(xd)
    J = torch.zeros(T, H, H, dtype=torch.float64, device="cuda")
    for e in range(E + shared):
        ws = [w[n][e] for n in ("w1", "w3", "w2")] if e < E else [w[n] for n in ("ws1", "ws3", "ws2")]
        t, k = torch.nonzero(idx == e, as_tuple=True) if e < E else (torch.arange(T, device="cuda"), None)
        if t.numel():
            ye, je, ve = mlp(xd[t], *[m.double() for m in ws])
            wt = gate[t, k].double()[:, None] if e < E else torch.ones(T, 1, dtype=torch.float64, device="cuda")
            exact.index_add_(0, t, wt * ye)
            J.index_add_(0, t, wt[..., None] * je)
            # the slot's output is held in fp16 before the sum
            var.index_add_(0, t, wt * wt * (ve + (ye * 2.0 ** -10) ** 2 / 12))
    sigma = check(y, exact, J, var, step(xd))
    assert 10 * sigma.mean() < exact.abs().mean()  # far below the outputs


@pytest.mark.parametrize("with_delta", [False, True])
def test_sublayer_and_capture(with_delta):
    T, H = 200, 256
    cfg, blk, w, g = block(T, 8, 2, H, 128, True, 2)
    gamma = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    draw = lambda: torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, delta = draw(), draw() if with_delta else None

    def want(x):
        total = x if delta is None else torch.empty_like(x)
        ffn = torch.empty_like(x)
        q, s = q8.add_rmsnorm(x, gamma, 1e-5, delta=delta, x_out=None if delta is None else total, y=ffn)
        blk2_q = q8.quantize(ffn)[0]  # the norm's own 8-bit rows come from the unrounded norm: near, not equal
        assert (blk2_q.int() - q.int()).abs().max() <= 1
        out, _ = blk.sublayer(x, gamma, delta=delta)
        return out.clone(), ffn, total

    y, ffn, total = want(x)
    got, x_ffn = blk.sublayer(x, gamma, delta=delta)
    assert torch.equal(got, y) and torch.equal(x_ffn, ffn)
    assert (y.float() - total.float()).abs().mean() > 0  # the mixture adds to the residual stream
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other, _ = blk.sublayer(x, gamma, delta=delta, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = blk.sublayer(x, gamma, delta=delta)
    for _ in range(3):
        x.copy_(draw())
        graph.replay()
        now = out.clone()
        assert torch.equal(now, blk.sublayer(x, gamma, delta=delta)[0])
    assert blk.device_error() == 0


def test_packed_weights_are_shared_and_bias_only_chooses():
    cfg, blk, w, g = block(64, 8, 2, 256, 128, True, 3)
    other = q8.MoeBlock(cfg, blk.w_router, blk.bias, None, None, None, packed=blk.weights)
    x = torch.randn(64, 256, generator=g, device="cuda").to(torch.bfloat16)
    assert torch.equal(blk(x), other(x))
    assert other.weights[0].data_ptr() == blk.weights[0].data_ptr()


@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (64, 512, 1024), (300, 256, 384), (1000, 768, 256)])
def test_dense_mlp(T, H, I):
    cfg, g = moe.Config.dense(T, H, I), gen(4)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").mul_(s[-1] ** -0.5).to(torch.bfloat16)  # noqa: E731
    w1, w3, w2 = draw(I, H), draw(I, H), draw(H, I)
    ffn = q8.DenseMlp(cfg, w1, w3, w2)
    wd = [m.double() for m in (w1, w3, w2)]
    for R in sorted({T, (T + 1) // 2, min(T, 65)}):  # one MLP serves fewer rows too
        x = torch.randn(R, H, generator=g, device="cuda").to(torch.bfloat16)
        res = torch.randn(R, H, generator=g, device="cuda").to(torch.bfloat16)
        y = ffn(x, residual=res)
        exact, J, var = mlp(x.double(), *wd)
        check(y, exact + res.double(), J, var, step(x.double()))
        assert torch.equal(ffn(x, residual=res, out=res), y)  # in place on the residual stream
    gamma = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    delta = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    y = ffn.sublayer(x, gamma, delta=delta)
    total = (x.double() + delta.double()).to(torch.bfloat16).double()
    n = total / torch.sqrt((total * total).mean(1, keepdim=True) + 1e-5) * gamma.double()
    exact, J, var = mlp(n, *wd)
    check(y, exact + total, J, var, step(n))
    with pytest.raises(ValueError):
        ffn(torch.cat([x, x]))
    assert ffn.device_error() == 0


def test_empty_batch_and_ids_out_of_range():
    cfg, blk, w, g = block(0, 4, 2, 256, 128, True, 5)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    assert blk(x).shape == (0, 256) and blk.device_error() == 0
    ffn = q8.DenseMlp(moe.Config.dense(8, 256, 128), w["ws1"], w["ws3"], w["ws2"])
    assert ffn(x).shape == (0, 256) and ffn.device_error() == 0
    # rows that are not finite come out not finite, and leave the others alone
    cfg, blk, w, g = block(64, 4, 2, 256, 128, True, 6)
    x = torch.randn(64, 256, generator=g, device="cuda").to(torch.bfloat16)
    good = blk(x).clone()
    gamma = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    sub = blk.sublayer(x, gamma)[0].clone()
    x[7, 3] = float("inf")
    x[9, 0] = float("nan")
    bad = blk.sublayer(x, gamma)[0]
    rest = [r for r in range(64) if r not in (7, 9)]
    assert torch.equal(bad[rest], sub[rest]) and torch.isnan(bad[[7, 9]]).all()
    x[7, 3] = x[9, 0] = 0
    assert not torch.isnan(good).any()
