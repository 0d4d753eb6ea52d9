"""Measured calls of the 8-bit expert path: rows to 8 bits (with the residual's addition and RMS norm), products of
8-bit integers with scales, dense and by expert, and rows sorted by expert and back with their gradients.

Shapes are those of the package's workloads (GLM-5 block: hidden 6144, expert width 2048, 256 experts, top 8, dense
width 12288; GLM-4.7-Flash: hidden 2048, expert width 1536, 64 experts, top 4) and generic ragged ones."""
import math

import torch

own = False  # True: run() calls the package; False: run() computes the plain form in 32 bits

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one token's pass through the norm before the experts: pure latency
        dict(name="norm one token", op="norm", T=1, H=6144, dtype="bf16", delta=True),
        # the prefill batch (4 x 4096 tokens): sum kept, normalised row for the router, 8-bit row for the experts
        dict(name="norm prefill", op="norm", T=16384, H=6144, dtype="bf16", delta=True),
        # hidden rows between the two products, a ragged batch whose rows are no multiple of 16 bytes
        dict(name="quantize ragged", op="quant", T=5003, H=1541, dtype="fp16", delta=False),
        # dense first-block MLP, up projection with SwiGLU, one token: the weights stream once
        dict(name="matmul one token", op="mm", R=1, N=24576, K=6144, swiglu=True, dtype="fp16", residual=False),
        # its down projection with the residual's addition at 64 decode tokens
        dict(name="matmul decode", op="mm", R=64, N=6144, K=12288, swiglu=False, dtype="bf16", residual=True),
        # ragged everything: rows, channels and reduction off every tile size, 32-bit results
        dict(name="matmul ragged", op="mm", R=777, N=1001, K=2064, swiglu=False, dtype="fp32", residual=False),
        # dense up projection of the prefill batch
        dict(name="matmul prefill", op="mm", R=16384, N=24576, K=6144, swiglu=True, dtype="fp16", residual=False),
        # expert up projection of 64 decode tokens: 256 experts with about two rows each and the shared one
        dict(name="experts decode", op="experts", T=64, E=256, top=8, N=4096, K=6144, swiglu=True, dtype="fp16"),
        # expert down projection of 4096 tokens over 64 experts
        dict(name="experts batch", op="experts", T=4096, E=64, top=4, N=2048, K=1536, swiglu=False, dtype="fp16"),
        # rows to the experts and back, 64 decode tokens
        dict(name="rows decode", op="rows", T=64, H=6144, E=256, top=8, dtype="bf16", ys="fp16"),
        # the same for the prefill batch
        dict(name="rows prefill", op="rows", T=16384, H=6144, E=256, top=8, dtype="bf16", ys="fp16"),
        # gradients of both directions for a training batch
        dict(name="rows gradient", op="rows_grad", T=4096, H=2048, E=64, top=4, dtype="bf16", ys="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "mm", "mm", "experts", "experts", "rows", "rows_grad"])
    if op in ("norm", "quant"):
        H = _log(rng, 64, 12288)
        H = H if rng.random() < 0.3 else (H + 7) // 8 * 8
        return dict(op=op, T=_log(rng, 1, 16384), H=H, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    delta=op == "norm" and rng.random() < 0.7)
    if op == "mm":
        swiglu = rng.random() < 0.4
        N = _log(rng, 96, 24576)
        return dict(op=op, R=_log(rng, 1, 8192), N=(N + 31) // 32 * 32 if swiglu else N,
                    K=(_log(rng, 128, 12288) + 15) // 16 * 16, swiglu=swiglu, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    residual=not swiglu and rng.random() < 0.5)
    if op == "experts":
        E = _log(rng, 2, 128)
        swiglu = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 4096), E=E, top=rng.randint(1, min(E, 8)),
                    N=(_log(rng, 128, 4096) + 31) // 32 * 32, K=(_log(rng, 128, 4096) + 15) // 16 * 16, swiglu=swiglu,
                    dtype=rng.choice(["bf16", "fp16"]))
    E = _log(rng, 2, 256)
    H = _log(rng, 64, 6144)
    return dict(op=op, T=_log(rng, 1, 8192), H=H if rng.random() < 0.3 else (H + 7) // 8 * 8, E=E,
                top=rng.randint(1, min(E, 8)), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                ys=rng.choice(["bf16", "fp16", "fp32"]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(g, rows, cols):
    """8-bit rows as quantised normal values leave them: about 127 at four standard deviations."""
    out = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    flat, step = out.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        v = torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.bfloat16)
        part.copy_(v.mul_(32).round_().clamp_(-127, 127))
    return out


def _scales(g, n, size):
    return (0.5 + torch.rand(n, generator=g, device="cuda")) * size


def _routing(g, T, E, top):
    """What the router and the permutation hand on: experts drawn without repetition with a skewed popularity,
    group offsets [E + 2] and the sorted row ids (a routed row t * top + slot; the shared expert's rows last)."""
    score = torch.rand((T, E), generator=g, device="cuda").log().neg().log().neg()
    score += torch.randn(E, generator=g, device="cuda") * 0.7
    idx = score.topk(top, dim=1).indices
    gate = torch.rand((T, top), generator=g, device="cuda") + 0.05
    gate = gate * 2.5 / gate.sum(1, keepdim=True)
    flat = idx.reshape(-1)
    ids = torch.cat([flat.argsort(stable=True), torch.arange(T * top, T * top + T, device="cuda")])
    counts = torch.bincount(flat, minlength=E)
    counts = torch.cat([counts, torch.full((1,), T, device="cuda")])
    offsets = torch.zeros(E + 2, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return gate, offsets, ids.to(torch.int32), int(counts[:E].max())


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    s = dict(case=case)
    if op in ("norm", "quant"):
        t = TYPES[c["dtype"]]
        x = torch.randn((c["T"], c["H"]), generator=g, device="cuda")
        x *= 1 + 8 * (torch.rand(c["H"], generator=g, device="cuda") < 0.01)  # a few loud channels
        s["x"] = x.to(t)
        if op == "norm":
            s["gamma"] = (1 + 0.1 * torch.randn(c["H"], generator=g, device="cuda")).to(t)
        if c["delta"]:
            s["delta"] = (0.5 * torch.randn((c["T"], c["H"]), generator=g, device="cuda")).to(t)
        return s
    if op in ("mm", "experts"):
        grouped = op == "experts"
        if grouped:
            _, s["offsets"], _, s["most"] = _routing(g, c["T"], c["E"], c["top"])
        R = c["T"] * (c["top"] + 1) if grouped else c["R"]
        G = c["E"] + 1 if grouped else 1
        s["x"], s["xs"] = _ints(g, R, c["K"]), _scales(g, R, 3.0 / 127)
        s["w"], s["ws"] = _ints(g, G * c["N"], c["K"]), _scales(g, G * c["N"], 0.08 / 127)
        if c.get("residual"):
            s["residual"] = torch.randn((R, c["N"]), generator=g, device="cuda").to(TYPES[c["dtype"]])
        if own:
            from sigmoid_routed_mixture_b200 import q8
            s["cfg"] = q8.MatmulConfig(R, c["N"], c["K"], groups=G, swiglu=c["swiglu"], dtype=TYPES[c["dtype"]])
            s["work"] = q8.workspace(s["cfg"])
        return s
    T, H, top, rows = c["T"], c["H"], c["top"], c["T"] * (c["top"] + 1)
    s["gate"], s["offsets"], s["sorted"], _ = _routing(g, T, c["E"], top)
    s["ys"] = torch.randn((rows, H), generator=g, device="cuda").to(TYPES[c["ys"]])
    if op == "rows":
        s["x"] = torch.randn((T, H), generator=g, device="cuda").to(TYPES[c["dtype"]])
    else:
        s["pos"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        s["pos"][s["sorted"].long()] = torch.arange(rows, dtype=torch.int32, device="cuda")
        s["dy"] = torch.randn((T, H), generator=g, device="cuda").to(TYPES[c["dtype"]])
        s["dxs"] = torch.randn((rows, H), generator=g, device="cuda").to(TYPES[c["dtype"]])
    if own:
        from sigmoid_routed_mixture_b200 import rows as R_
        s["cfg"] = R_.Config(T, H, c["E"], top, dtype=TYPES[c["dtype"]], slot_dtype=TYPES[c["ys"]])
        s["work"] = R_.workspace()
    return s


# ------------------------------------------------------------------ one pass

def _value_type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _run_own(s):
    from sigmoid_routed_mixture_b200 import q8, rows
    c, op = s["case"], s["case"]["op"]
    if op == "quant":
        q, scale = q8.quantize(s["x"])
        return dict(values=q8.dequantize(q, scale, _value_type(c)), scale=scale)
    if op == "norm":
        x, y = s["x"], torch.empty_like(s["x"])
        total = torch.empty_like(x) if c["delta"] else None
        q, scale = q8.add_rmsnorm(x, s["gamma"], EPS, delta=s.get("delta"), x_out=total, y=y)
        out = dict(values=q8.dequantize(q, scale, _value_type(c)), scale=scale, norm=y)
        return dict(out, total=total) if c["delta"] else out
    if op in ("mm", "experts"):
        return q8.matmul(s["cfg"], s["x"], s["xs"], s["w"], s["ws"], s["work"], offsets=s.get("offsets"),
                         residual=s.get("residual"))
    if op == "rows":
        xs, pos = rows.sort(s["cfg"], s["x"], s["offsets"], s["sorted"], s["work"])
        return dict(xs=xs, pos=pos, y=rows.unsort(s["cfg"], s["ys"], s["gate"], pos, s["work"]))
    dys, dgate = rows.unsort_grad(s["cfg"], s["dy"], s["ys"], s["gate"], s["pos"], s["work"])
    return dict(dys=dys, dgate=dgate, dx=rows.sort_grad(s["cfg"], s["dxs"], s["pos"], s["work"]))


def _swiglu(z):
    """Columns in units of 32, 16 gate channels and then the 16 matching up channels."""
    u = z.view(*z.shape[:-1], z.shape[-1] // 32, 2, 16)
    gate, up = u[..., 0, :], u[..., 1, :]
    return (gate / (1 + torch.exp(-gate)) * up).reshape(*z.shape[:-1], z.shape[-1] // 2)


def run(s):
    if own:
        return _run_own(s)
    c, op = s["case"], s["case"]["op"]
    if op in ("norm", "quant"):
        t = TYPES[c["dtype"]]
        x = s["x"]
        if c["delta"]:
            x = (x.float() + s["delta"].float()).to(t)
        n = x.float()
        if op == "norm":
            n = n / torch.sqrt((n * n).mean(1, keepdim=True) + EPS) * s["gamma"].float()
        scale = n.abs().amax(1) / 127
        q = torch.round(n / scale[:, None])
        out = dict(values=(q * scale[:, None]).to(_value_type(c)), scale=scale)
        if op == "norm":
            out["norm"] = n.to(t)
        if c["delta"]:
            out["total"] = x
        return out
    if op == "mm":
        z = (s["x"].float() @ s["w"].float().t()) * s["xs"][:, None] * s["ws"]
        z = _swiglu(z) if c["swiglu"] else z
        return (z + s["residual"].float() if c.get("residual") else z).to(TYPES[c["dtype"]])
    if op == "experts":
        # the routed groups padded to the largest one's rows in one batched product, the shared group by itself
        E, N, T, t = c["E"], c["N"], c["T"], TYPES[c["dtype"]]
        R = T * c["top"]
        first, last = s["offsets"][:E, None], s["offsets"][1:E + 1, None]
        at = first + torch.arange(s["most"], device="cuda")
        real = at < last
        at = torch.where(real, at, 0).long()
        w, ws = s["w"].view(E + 1, N, -1), s["ws"].view(E + 1, 1, N)
        z = torch.bmm(s["x"][at].float(), w[:E].float().transpose(1, 2)) * s["xs"][at][..., None] * ws[:E]
        zs = (s["x"][R:].float() @ w[E].float().t()) * s["xs"][R:, None] * ws[E]
        if c["swiglu"]:
            z, zs = _swiglu(z), _swiglu(zs)
        out = torch.empty((R + 1 + T, z.shape[-1]), dtype=t, device="cuda")
        out[torch.where(real, at, R + T)] = z.to(t)  # padding goes to one row more
        out[R:R + T] = zs.to(t)
        return out[:R + T]
    T, top, H = c["T"], c["top"], c["H"]
    tk = T * top
    if op == "rows":
        ids = s["sorted"].long()
        xs = s["x"][torch.where(ids < tk, ids // top, ids - tk)]
        pos = torch.empty(ids.numel(), dtype=torch.int32, device="cuda")
        pos[ids] = torch.arange(ids.numel(), dtype=torch.int32, device="cuda")
        p = pos.long()
        y = (s["gate"][..., None] * s["ys"][p[:tk]].view(T, top, H).float()).sum(1) + s["ys"][p[tk:]].float()
        return dict(xs=xs, pos=pos, y=y.to(TYPES[c["dtype"]]))
    p, dy = s["pos"].long(), s["dy"].float()
    dgate = (s["ys"][p[:tk]].view(T, top, H).float() * dy[:, None]).sum(2)
    dys = torch.empty_like(s["ys"])
    dys[p[:tk]] = (s["gate"][..., None] * dy[:, None]).view(tk, H).to(dys.dtype)
    dys[p[tk:]] = dy.to(dys.dtype)
    dx = s["dxs"][p[:tk]].view(T, top, H).float().sum(1) + s["dxs"][p[tk:]].float()
    return dict(dys=dys, dgate=dgate, dx=dx.to(TYPES[c["dtype"]]))


# ------------------------------------------------------------------ floors

def work(case):
    c, op = case, case["op"]
    size = lambda t: TYPES[t].itemsize  # noqa: E731
    if op in ("norm", "quant"):
        n, e = c["T"] * c["H"], size(c["dtype"])
        b = n * e + n * 2 + 4 * c["T"]  # rows in, the 8-bit rows' values and scales out
        b += (n * e + c["H"] * e) if op == "norm" else 0  # the normalised rows out, gamma in
        return dict(bytes=b + (2 * n * e if c["delta"] else 0), flops=8 * n)
    if op in ("mm", "experts"):
        grouped = op == "experts"
        R = c["T"] * (c["top"] + 1) if grouped else c["R"]
        # experts with at least one row: all but those that every token passes over, were the choice uniform
        G = 1 + c["E"] * (1 - (1 - c["top"] / c["E"]) ** c["T"]) if grouped else 1
        y = R * (c["N"] // 2 if c["swiglu"] else c["N"]) * size(c["dtype"])
        b = R * (c["K"] + 4) + G * c["N"] * (c["K"] + 4) + y * (2 if c.get("residual") else 1)
        return dict(bytes=b, flops=2 * R * c["N"] * c["K"])
    T, H, rows, e, es = c["T"], c["H"], c["T"] * (c["top"] + 1), size(c["dtype"]), size(c["ys"])
    if op == "rows":
        b = T * H * e + rows * H * e + rows * 8 + rows * H * es + T * H * e + 4 * T * c["top"]
        return dict(bytes=b, flops=2 * rows * H)
    b = T * H * e + 2 * rows * H * es + 8 * T * c["top"] + 4 * rows + rows * H * e + T * H * e
    return dict(bytes=b, flops=4 * rows * H)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op in ("norm", "quant"):
        x = s["x"].double()
        if c["delta"]:
            x = (x + s["delta"].double()).to(s["x"].dtype).double()
        n, out = x, {}
        if op == "norm":
            mean = torch.einsum("th,th->t", x, x) / c["H"]
            n = torch.einsum("th,t,h->th", x, (mean + EPS).rsqrt(), s["gamma"].double())
            out["norm"] = n
        scale = torch.maximum(n.amax(1), -n.amin(1)).div(127)
        out.update(values=n.div(scale.unsqueeze(1)).round().mul(scale.unsqueeze(1)), scale=scale)
        if c["delta"]:
            out["total"] = x
        return out

    def product(x, xs, w, ws):
        z = torch.einsum("rk,nk->rn", x.double(), w.double())
        z = torch.einsum("rn,r,n->rn", z, xs.double(), ws.double())
        if c["swiglu"]:
            pairs = z.unflatten(1, (-1, 32))
            a, b = pairs[..., :16].flatten(1), pairs[..., 16:].flatten(1)
            z = a * torch.sigmoid(a) * b
        return z

    if op == "mm":
        z = product(s["x"], s["xs"], s["w"], s["ws"])
        return z + s["residual"].double() if c.get("residual") else z
    if op == "experts":
        edges, parts = s["offsets"].tolist(), []
        for g, (a, b) in enumerate(zip(edges, edges[1:])):
            w = slice(g * c["N"], (g + 1) * c["N"])
            if b > a:
                parts.append(product(s["x"][a:b], s["xs"][a:b], s["w"][w], s["ws"][w]))
        return torch.cat(parts)
    T, top = c["T"], c["top"]
    ids = s["sorted"].long()
    place = torch.argsort(ids)  # row id -> sorted position
    routed, shared = place[: T * top].view(T, top), place[T * top:]
    if op == "rows":
        y = s["ys"][shared].double()
        for k in range(top):
            y += s["gate"][:, k:k + 1].double() * s["ys"][routed[:, k]].double()
        token = torch.cat([torch.arange(T, device="cuda").repeat_interleave(top), torch.arange(T, device="cuda")])
        return dict(xs=s["x"][token[ids]], pos=None, y=y)
    dy = s["dy"].double()
    dgate = torch.stack([torch.einsum("th,th->t", dy, s["ys"][routed[:, k]].double()) for k in range(top)], 1)
    weight = torch.cat([s["gate"].double().flatten(), torch.ones(T, dtype=torch.float64, device="cuda")])
    token = torch.cat([torch.arange(T, device="cuda").repeat_interleave(top), torch.arange(T, device="cuda")])
    dys = dy[token[ids]].mul_(weight[ids, None])
    dx = s["dxs"][shared].double()
    for k in range(top):
        dx += s["dxs"][routed[:, k]].double()
    return dict(dys=dys, dgate=dgate, dx=dx)
