"""Cases that measure the 8-bit forward pass of a Mixture-of-Experts layer and the router's losses: root-mean-square
norm with the residual's addition and an 8-bit output, its gradient, the experts' weights in 8 bits, the per-expert
product in 8-bit floating point with a scale for each block of 128 (plain, and with the SwiGLU activation back in 8
bits), and the balance and z losses of the router with the gradient of its logits.

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits; with ``own`` true it makes the
calls of this repository's package.  ``exact`` states each operator once more in 64 bits.  8-bit results come as their
e4m3 codes, each block's scale beside them.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
BLOCK = 128          # columns (and, of weights, rows) that share one scale
TOP = 448.0          # largest e4m3 value
TINY = 2.0 ** -117   # blocks below it are stored as zeros
EPS = 1e-5


def listed():
    return [
        # a decode batch: experts' sum added to the residual stream, normed for the router (bf16) and the experts (8 bits)
        dict(name="rmsnorm_decode", op="rmsnorm", T=64, d=4096, x="f32", h="bf16", out="both"),
        # the same step for a prompt batch of the Mixtral-shaped layer
        dict(name="rmsnorm_mixtral", op="rmsnorm", T=8192, d=4096, x="f32", h="bf16", out="both"),
        # a small training batch of odd size, fp32 residual stream: the gradient at latency-bound size
        dict(name="rmsnorm_backward_small", op="rmsnorm_backward", T=333, d=2064, h="f32", dy="f32"),
        # the norm before the Mixtral-shaped layer in training
        dict(name="rmsnorm_backward_mixtral", op="rmsnorm_backward", T=8192, d=4096, h="bf16", dy="f32"),
        # the tiny layer's weights, laid out for the 8-bit product
        dict(name="quantize_tiny", op="quantize", E=8, d=512, N=1024, halves=1),
        # the gate and up projections of the fine-grained layer (F = 1408) when a model is loaded
        dict(name="quantize_finegrained", op="quantize", E=64, d=2048, N=2816, halves=2),
        # down projection of a decode batch, four hot experts of 128: the weights' bytes
        dict(name="fp8_gemm_decode", op="fp8_gemm", T=64, d=1536, E=128, k=8, N=4096, load="hot4", gather=False, out="bf16"),
        # down projection of the Mixtral-shaped layer: tensor-core work
        dict(name="fp8_gemm_mixtral", op="fp8_gemm", T=8192, d=14336, E=8, k=2, N=4096, load="none", gather=False, out="bf16"),
        # the tiny layer's gate and up projections from token rows: latency
        dict(name="fp8_swiglu_tiny", op="fp8_swiglu", T=256, d=512, E=8, k=2, F=512, load="none", gather=True),
        # gate and up projections of the fine-grained layer, Zipf load, experts without rows
        dict(name="fp8_swiglu_finegrained", op="fp8_swiglu", T=16384, d=2048, E=64, k=4, F=1408, load="zipf", gather=True),
        # router of the fine-grained layer for an odd batch with padding rows: latency
        dict(name="router_losses_small", op="router_losses", T=333, E=64, k=4, gates="renorm", seq=0, masked=True),
        # router of the DeepSeek-V3-shaped layer: logistic gates, the loss taken for each sequence of 2048 tokens
        dict(name="router_losses_deepseek_v3", op="router_losses", T=32768, E=256, k=8, gates="sigmoid_renorm", seq=2048,
             masked=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step=16):
    return max(lo, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(("rmsnorm", "rmsnorm_backward", "quantize", "fp8_gemm", "fp8_swiglu", "router_losses"))
    ty = lambda: rng.choice(("f32", "bf16"))  # noqa: E731
    if op in ("rmsnorm", "rmsnorm_backward"):
        d = _width(rng, 64, 16384)
        c = dict(op=op, T=_log_int(rng, 1, min(32768, (1 << 27) // d)), d=d, h=ty())
        return dict(c, dy=ty()) if op == "rmsnorm_backward" else dict(c, x=ty(), out=rng.choice(("y", "codes", "both")))
    if op == "quantize":
        while True:
            halves = rng.randint(1, 2)
            c = dict(op=op, E=_log_int(rng, 1, 256), d=_width(rng, 64, 8192), N=_width(rng, 64, 16384, 16 * halves),
                     halves=halves)
            if c["E"] * c["d"] * c["N"] <= 1 << 29:
                return c
    if op == "router_losses":
        E = _log_int(rng, 1, 1024)
        return dict(op=op, T=_log_int(rng, 1, min(65536, (1 << 24) // E)), E=E, k=rng.randint(1, min(8, E)),
                    gates=rng.choice(("softmax", "renorm", "sigmoid", "sigmoid_renorm")),
                    seq=rng.choice((0, 0, _log_int(rng, 1, 8192))), masked=rng.choice((True, False)))
    while True:
        E = _log_int(rng, 1, 256)
        c = dict(op=op, T=_log_int(rng, 1, 16384), d=_width(rng, 64, 14336), E=E, k=rng.randint(1, min(8, E)),
                 load=rng.choice(("none", "zipf")), gather=rng.choice((True, False)))
        N = _width(rng, 64, 16384)
        if op == "fp8_gemm":
            c.update(N=N, out=ty())
        else:
            N = N // 32 * 32
            c.update(F=N // 2)
        if c["T"] * c["k"] * c["d"] * N <= 9e11 and E * c["d"] * N <= 1 << 29:
            return c


def _blocks(n):
    return -(-n // BLOCK)


def _experts_with_rows(c):
    """Expected number of experts that receive a row (hot4: four experts hold half of the picks)."""
    E, S = c["E"], c["T"] * c["k"]
    if c["load"] == "hot4":
        return 4 + (E - 4) * (1 - math.exp(-(S - 4 * c["T"]) / (E - 4)))
    if c["load"] == "zipf":
        p = [(r + 1) ** -1.1 for r in range(E)]
        live = max(E - 4 if E > 4 else E, c["k"])  # the four least popular get no row
        return sum(1 - math.exp(-min(S * p[r] / sum(p), c["T"])) for r in range(live))
    return E * (1 - math.exp(-S / E))


def work(c):
    size = {"f32": 4, "bf16": 2}
    op = c["op"]
    if op == "rmsnorm":  # x and the residual in; the sum, the normed rows and the row's 1 / rms out
        T, d = c["T"], c["d"]
        b = T * d * (size[c["x"]] + 2 * size[c["h"]]) + 4 * T + 4 * d
        b += T * d * 2 if c["out"] != "codes" else 0
        b += T * (d + 4 * _blocks(d)) if c["out"] != "y" else 0
        return dict(bytes=b, flops=6 * T * d)
    if op == "rmsnorm_backward":
        T, d = c["T"], c["d"]
        return dict(bytes=T * d * (3 * size[c["h"]] + size[c["dy"]]) + 4 * T + 8 * d, flops=10 * T * d)
    if op == "quantize":
        n = c["E"] * c["d"] * c["N"]
        return dict(bytes=3 * n + 4 * n // (BLOCK * BLOCK), flops=2 * n)
    if op == "router_losses":  # forward reads logits and picks, backward the same again and writes the gradient
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=T * E * 12 + T * k * 12 + 2 * T, flops=16 * T * E)
    T, k, d, E = c["T"], c["k"], c["d"], c["E"]
    S, N = T * k, c.get("N") or 2 * c["F"]
    rows = T if c["gather"] else S
    b = rows * (d + 4 * _blocks(d)) + _experts_with_rows(c) * d * N
    b += S * N * size[c["out"]] if op == "fp8_gemm" else S * (c["F"] + 4 * _blocks(c["F"]))
    return dict(bytes=b, flops=2 * S * d * N)


# ---------------------------------------------------------------- inputs

def _routing(c, g, dev):
    """Expert of every routed slot, as a router gives it: T tokens, k different experts each."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn(T, E, generator=g, device=dev)
    order = torch.randperm(E, generator=g, device=dev)
    if c["load"] == "zipf":
        p = torch.arange(1, E + 1, device=dev, dtype=torch.float32) ** -1.1
        p = torch.log(p / p.sum())
        if E > 4:
            p[max(E - 4, k):] = -30.0
        logits[:, order] += p
    elif c["load"] == "hot4":
        logits[:, order[:4]] += 16.0
    return torch.topk(logits, k, dim=1).indices


def _activations(shape, g, dev, dtype, scale=1.0):
    """Normal values with a few wide channels, as hidden activations have."""
    v = torch.randn(shape, generator=g, device=dev)
    wide = torch.randint(0, shape[-1], (max(1, shape[-1] // 256),), generator=g, device=dev)
    v[..., wide] *= 6.0
    return v.mul_(scale).to(dtype)


def _codes(shape, g, dev):
    """e4m3 codes spread as those of normal values under their block's largest magnitude."""
    out = torch.empty(shape, dtype=E4M3, device=dev)
    flat = out.view(-1)
    step = 1 << 26
    parts = [flat[i:i + step] for i in range(0, flat.numel(), step)]
    [p.copy_(torch.randn(p.numel(), generator=g, device=dev).mul_(150.0).clamp_(-TOP, TOP)) for p in parts]
    return out


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"c": c}
    op = c["op"]

    def normal(shape, dtype=torch.float32, scale=1.0):
        return torch.randn(shape, generator=g, device=dev).mul_(scale).to(dtype)

    def scales(shape, typical):
        return torch.exp(normal(shape, scale=0.3)).mul_(typical / 150.0)

    if op == "rmsnorm":
        T, d = c["T"], c["d"]
        s["x"] = normal((T, d), DTYPES[c["x"]], 0.5)
        s["res"] = _activations((T, d), g, dev, DTYPES[c["h"]])
        s["gamma"] = 1.0 + normal((d,), scale=0.1)
    elif op == "rmsnorm_backward":
        T, d = c["T"], c["d"]
        s["h"] = _activations((T, d), g, dev, DTYPES[c["h"]])
        s["gamma"] = 1.0 + normal((d,), scale=0.1)
        s["rstd"] = (1.0 / torch.sqrt(s["h"].double().square().mean(1) + EPS)).float()
        s["dy"] = normal((T, d), DTYPES[c["dy"]], 1e-2)
        s["dres"] = normal((T, d), DTYPES[c["h"]], 1e-2)
    elif op == "quantize":
        E, d, N = c["E"], c["d"], c["N"]
        s["W"] = torch.empty(E, d, N, dtype=torch.bfloat16, device=dev)
        [s["W"][e].copy_(normal((d, N), scale=1.0 / math.sqrt(d))) for e in range(E)]
    elif op == "router_losses":
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = normal((T, E)) + normal((E,), scale=0.5)
        s["topk_idx"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
        s["dw"] = normal((T, k), scale=1e-2)
        # padding at the end of about a third of the sequences, and whole sequences of nothing else
        s["mask"] = None
        if c["masked"]:
            L = c["seq"] or T
            n = -(-T // L)
            live = torch.rand(n, generator=g, device=dev)
            live = torch.where(live < 0.05, torch.zeros_like(live), torch.clamp(live * 3.0, max=1.0))
            if n == 1:
                live.clamp_(min=0.5)
            t = torch.arange(T, device=dev)
            s["mask"] = (t % L) < (live * L).ceil()[t // L]
    else:
        T, k, d, E = c["T"], c["k"], c["d"], c["E"]
        S, N = T * k, c.get("N") or 2 * c["F"]
        idx = _routing(c, g, dev).reshape(-1)
        counts = torch.bincount(idx, minlength=E)
        s["counts"] = counts.tolist()  # the plain form's slices
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["perm"] = torch.argsort(idx, stable=True).to(torch.int32) if c["gather"] else None
        rows = T if c["gather"] else S
        s["A"], s["As"] = _codes((rows, d), g, dev), scales((rows, _blocks(d)), 1.0)
        nb = _blocks(N) if op == "fp8_gemm" else 2 * _blocks(c["F"])
        s["W"], s["Ws"] = _codes((E, N, d), g, dev), scales((E, nb, _blocks(d)), 1.0 / math.sqrt(d))
    if own:
        _handles(s, dev)
    return s


_FLAGS = {"softmax": 0, "renorm": 1, "sigmoid": 2, "sigmoid_renorm": 3}
BALANCE, Z = 1e-2, 1e-3


def _handles(s, dev):
    """The plan, workspace and result buffers that a program of this package keeps."""
    from moe_token_dispatch_route_gb300 import binding
    s["api"] = binding
    c, op = s["c"], s["c"]["op"]
    f32, bf16 = torch.float32, torch.bfloat16
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
    if op == "rmsnorm":
        T, d = c["T"], c["d"]
        s["plan"] = binding.moe_plan(T, d, 1, 1, 256)
        s["h"], s["rstd"] = new((T, d), DTYPES[c["h"]]), new((T,), f32)
        s["y"] = new((T, d), bf16) if c["out"] != "codes" else None
        s["codes"] = new((T, d), E4M3) if c["out"] != "y" else None
        s["scales"] = new((T, _blocks(d)), f32) if c["out"] != "y" else None
    elif op == "rmsnorm_backward":
        T, d = c["T"], c["d"]
        s["plan"] = binding.moe_plan(T, d, 1, 1, 256)
        s["dx"], s["dgamma"] = new((T, d), DTYPES[c["h"]]), new((d,), f32)
        s["scratch"] = binding.backward_scratch(s["plan"])
    elif op == "quantize":
        E, d, N, halves = c["E"], c["d"], c["N"], c["halves"]
        s["plan"] = binding.moe_plan(1, d, E, 1, N)
        s["codes"], s["scales"] = new((E, N, d), E4M3), new((E, halves * _blocks(N // halves), _blocks(d)), f32)
    elif op == "router_losses":
        T, E, k = c["T"], c["E"], c["k"]
        s["plan"] = binding.moe_plan(T, 256, E, k, 256, route_flags=_FLAGS[c["gates"]])
        groups = -(-T // c["seq"]) if c["seq"] else 1
        s["loss"], s["load"] = new((2,), f32), new((groups, E), torch.int32)
        s["tokens"], s["dlogits"] = new((groups + 1,), torch.int32), new((T, E), f32)
        s["scratch"] = binding.balance_scratch(s["plan"], c["seq"])
    else:
        T, k, d, E = c["T"], c["k"], c["d"], c["E"]
        S = T * k
        if op == "fp8_gemm":
            out = binding.MOE_OUT_BF16 if c["out"] == "bf16" else binding.MOE_OUT_F32
            s["plan"] = binding.moe_plan(T, d, E, k, c["N"], out_dtype=out)
            s["Y"] = new((S, c["N"]), DTYPES[c["out"]])
        else:
            F = c["F"]
            s["plan"] = binding.moe_plan(T, d, E, k, 2 * F)
            s["H"], s["Hs"] = new((S, F), E4M3), new((S, _blocks(F)), f32)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device=dev)
        s["status"] = torch.zeros(4, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _PLAIN[state["c"]["op"]](state)


def _given(**kw):
    return {k: v for k, v in kw.items() if v is not None}


def _run_own(s):
    b, c, plan = s["api"], s["c"], s["plan"]
    op = c["op"]
    if op == "rmsnorm":
        b.moe_rmsnorm(plan, s["x"], s["res"], s["gamma"], EPS, s["h"], s["y"], s["codes"], s["scales"], s["rstd"])
        return _given(h=s["h"], y=s["y"], codes=s["codes"], scales=s["scales"], rstd=s["rstd"])
    if op == "rmsnorm_backward":
        b.moe_rmsnorm_backward(plan, s["dy"], s["h"], s["gamma"], s["rstd"], s["dres"], s["dx"], s["dgamma"], s["scratch"])
        return {"dx": s["dx"], "dgamma": s["dgamma"]}
    if op == "quantize":
        b.moe_quantize_weights(plan, s["W"], s["codes"], s["scales"], c["halves"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "router_losses":
        b.moe_balance_loss(plan, s["logits"], s["topk_idx"], s["mask"], c["seq"], BALANCE, Z, s["loss"], s["load"],
                           s["tokens"], s["scratch"])
        b.moe_router_backward(plan, s["logits"], s["topk_idx"], s["dw"], s["mask"], c["seq"], BALANCE, Z, s["load"],
                              s["tokens"], s["dlogits"])
        return {"loss": s["loss"], "load": s["load"], "tokens": s["tokens"], "dlogits": s["dlogits"]}
    if op == "fp8_gemm":
        b.moe_grouped_gemm_fp8(plan, s["A"], s["As"], s["perm"], s["offsets"], s["W"], s["Ws"], s["Y"], s["workspace"],
                               s["status"])
        return {"Y": s["Y"]}
    b.moe_grouped_gemm_fp8_swiglu(plan, s["A"], s["As"], s["perm"], s["offsets"], s["W"], s["Ws"], s["H"], s["Hs"],
                                  s["workspace"], s["status"])
    return {"H": s["H"], "scales": s["Hs"]}


def _padded(v, n):
    """[rows, n] in blocks of 128, the last one filled up with zeros."""
    return torch.nn.functional.pad(v, (0, _blocks(n) * BLOCK - n)).reshape(v.shape[0], _blocks(n), BLOCK)


def _store(v):
    """e4m3 codes and fp32 scales of rows: scale = amax / 448, code = nearest even of v * (448 / amax)."""
    n = v.shape[1]
    b = _padded(v, n)
    amax = b.abs().amax(-1, keepdim=True)
    live = amax >= TINY
    amax = torch.where(live, amax, 1.0)
    codes = torch.where(live, b * (TOP / amax), 0.0).to(E4M3).reshape(v.shape[0], -1)[:, :n].contiguous()
    return codes, torch.where(live, amax / TOP, 0.0)[:, :, 0].contiguous()


def _rmsnorm(s):
    c = s["c"]
    h = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(1) + EPS)
    y = hf * rstd[:, None] * s["gamma"]
    codes, scales = _store(y) if c["out"] != "y" else (None, None)
    return _given(h=h, y=y.to(torch.bfloat16) if c["out"] != "codes" else None, codes=codes, scales=scales, rstd=rstd)


def _rmsnorm_backward(s):
    dy, r = s["dy"].float(), s["rstd"][:, None]
    hh = s["h"].float() * r
    v = dy * s["gamma"]
    dx = r * (v - hh * (v * hh).mean(1, keepdim=True)) + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dgamma": (dy * hh).sum(0)}


def _tiles(w, halves):
    """[E, d, N] as [E, halves, column blocks, 128, row blocks, 128] of the transposed weights, padded with zeros."""
    E, d, N = w.shape
    n = N // halves
    t = w.reshape(E, d, halves, n).permute(0, 2, 3, 1)
    t = torch.nn.functional.pad(t, (0, _blocks(d) * BLOCK - d, 0, _blocks(n) * BLOCK - n))
    return t.reshape(E, halves, _blocks(n), BLOCK, _blocks(d), BLOCK)


def _quantize(s):
    E, d, N = s["W"].shape
    halves = s["c"]["halves"]
    t = _tiles(s["W"].float(), halves)
    amax = t.abs().amax((3, 5), keepdim=True)
    live = amax >= TINY
    amax = torch.where(live, amax, 1.0)
    n = N // halves
    codes = torch.where(live, t * (TOP / amax), 0.0).to(E4M3)
    codes = codes.reshape(E, halves, _blocks(n) * BLOCK, -1)[:, :, :n, :d].reshape(E, N, d).contiguous()
    return {"codes": codes, "scales": torch.where(live, amax / TOP, 0.0).reshape(E, halves * _blocks(n), _blocks(d)).contiguous()}


def _scores(logits, gates):
    if gates.startswith("sigmoid"):
        return 1.0 / (1.0 + torch.exp(-logits))
    m = logits.amax(1, keepdim=True)
    e = torch.exp(logits - m)
    return e / e.sum(1, keepdim=True)


def _router_losses(s):
    c = s["c"]
    T, E, k = c["T"], c["E"], c["k"]
    L = c["seq"] or T
    G = -(-T // L)
    logits, dev = s["logits"].double(), s["logits"].device  # sums over all tokens
    live = s["mask"].double() if s["mask"] is not None else torch.ones(T, dtype=torch.float64, device=dev)
    idx = s["topk_idx"].long()
    group = torch.arange(T, device=dev) // L
    picks = torch.zeros(T, E, dtype=torch.float64, device=dev).scatter_(1, idx, 1.0)
    load = torch.zeros(G, E, dtype=torch.float64, device=dev).index_add_(0, group, picks * live[:, None])
    n = torch.zeros(G, dtype=torch.float64, device=dev).index_add_(0, group, live)
    score = _scores(logits, c["gates"])
    total = score.sum(1, keepdim=True)
    p = score / total  # the softmax's are 1 in sum already
    psum = torch.zeros(G, E, dtype=torch.float64, device=dev).index_add_(0, group, p * live[:, None])
    a = torch.where(n > 0, BALANCE * E / (G * k * torch.where(n > 0, n, 1.0) ** 2), 0.0)
    m = logits.amax(1, keepdim=True)
    lse = m[:, 0] + torch.log(torch.exp(logits - m).sum(1))
    counted = torch.clamp(n.sum(), min=1.0)
    loss = torch.stack([(a[:, None] * load * psum).sum(), Z * (lse.square() * live).sum() / counted])
    w = (a[:, None] * load)[group]
    d = p * (w - (p * w).sum(1, keepdim=True)) * live[:, None]
    if c["gates"].startswith("sigmoid"):
        d = d * (1.0 - score)
    d = d + (2.0 * Z / counted * lse * live)[:, None] * torch.exp(logits - lse[:, None])
    picked = score.gather(1, idx)
    dw = s["dw"].double()
    if c["gates"] == "softmax":
        d = d - score * (picked * dw).sum(1, keepdim=True)
        dl = picked * dw
    elif c["gates"] == "sigmoid":
        dl = dw * picked * (1.0 - picked)
    else:
        g = picked / picked.sum(1, keepdim=True)
        dl = g * (dw - (g * dw).sum(1, keepdim=True))
        if c["gates"] == "sigmoid_renorm":
            dl = dl * (1.0 - picked)
    d.scatter_add_(1, idx, dl)
    tokens = torch.cat([n, n.sum(0, keepdim=True)]).to(torch.int32)
    return {"loss": loss.float(), "load": load.to(torch.int32), "tokens": tokens, "dlogits": d.float()}


def _rows(s):
    """The product's rows in expert order, in 32 bits: code times scale, zeros up to whole blocks."""
    d = s["A"].shape[1]
    v = _padded(s["A"].float(), d) * s["As"][:, :, None]
    v = v.reshape(v.shape[0], -1)[:, :d]
    return v if s["perm"] is None else v[(s["perm"] // s["c"]["k"]).long()]


def _weights(s, e, halves):
    """[N, d] of one expert in 32 bits."""
    N, d = s["W"].shape[1:]
    n = N // halves
    row = torch.arange(N, device=s["W"].device)
    row = row // n * _blocks(n) + row % n // BLOCK
    col = torch.arange(d, device=s["W"].device) // BLOCK
    return s["W"][e].float() * s["Ws"][e][row][:, col]


def _product(s, halves):
    parts = torch.split(_rows(s), s["counts"])
    return torch.cat([p @ _weights(s, e, halves).T for e, p in enumerate(parts) if s["counts"][e]])


def _fp8_gemm(s):
    return {"Y": _product(s, 1).to(DTYPES[s["c"]["out"]])}


def _fp8_swiglu(s):
    F = s["c"]["F"]
    gu = _product(s, 2)
    g = gu[:, :F]
    H, scales = _store(g / (1.0 + torch.exp(-g)) * gu[:, F:])
    return {"H": H, "scales": scales}


_PLAIN = {"rmsnorm": _rmsnorm, "rmsnorm_backward": _rmsnorm_backward, "quantize": _quantize, "fp8_gemm": _fp8_gemm,
          "fp8_swiglu": _fp8_swiglu, "router_losses": _router_losses}


# ---------------------------------------------------------------- 64 bits

def _scaled(v):
    """A row's values over its blocks' scales, before they are rounded to 8 bits, and the scales."""
    codes, scales = [], []
    for c0 in range(0, v.shape[1], BLOCK):
        b = v[:, c0:c0 + BLOCK]
        scale = b.abs().max(1, keepdim=True).values / TOP
        scales.append(scale)
        codes.append(torch.where(scale > 0, b / torch.where(scale > 0, scale, 1.0), 0.0))
    return torch.cat(codes, 1), torch.cat(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "rmsnorm":
        # the sum is rounded to 32 bits and then to the residual's type, and the norm is of what is stored
        h = (s["x"].double() + s["res"].double()).float().to(s["res"].dtype).double()
        rstd = (torch.einsum("td,td->t", h, h) / c["d"] + EPS) ** -0.5
        y = torch.einsum("td,t,d->td", h, rstd, s["gamma"].double())
        codes, scales = _scaled(y) if c["out"] != "y" else (None, None)
        return _given(h=h, y=y if c["out"] != "codes" else None, codes=codes, scales=scales, rstd=rstd)
    if op == "rmsnorm_backward":
        # dx = (r - r^3 h h' / d) (gamma dy) + dres
        h, r, dy = s["h"].double(), s["rstd"].double(), s["dy"].double()
        v = dy * s["gamma"].double()
        dx = r[:, None] * v - (r ** 3 / c["d"] * torch.einsum("td,td->t", v, h))[:, None] * h + s["dres"].double()
        return {"dx": dx, "dgamma": torch.einsum("td,td,t->d", dy, h, r)}
    if op == "quantize":
        E, d, N, halves = c["E"], c["d"], c["N"], c["halves"]
        n = N // halves
        codes = torch.empty(E, N, d, dtype=torch.float64, device=s["W"].device)
        scales = torch.empty(E, halves * _blocks(n), _blocks(d), dtype=torch.float64, device=s["W"].device)
        for half in range(halves):
            for i in range(_blocks(n)):
                r0, r1 = half * n + i * BLOCK, half * n + min(n, (i + 1) * BLOCK)
                w = s["W"][:, :, r0:r1].double().transpose(1, 2)
                for j in range(_blocks(d)):
                    b = w[:, :, j * BLOCK:(j + 1) * BLOCK]
                    scale = b.abs().amax((1, 2)) / TOP
                    scales[:, half * _blocks(n) + i, j] = scale
                    codes[:, r0:r1, j * BLOCK:(j + 1) * BLOCK] = b / torch.where(scale > 0, scale, 1.0)[:, None, None]
        return {"codes": codes, "scales": scales}
    if op == "router_losses":
        return _exact_router(s)
    gu = _exact_product(s, 1 if op == "fp8_gemm" else 2)
    if op == "fp8_gemm":
        return {"Y": gu}
    g, u = gu.chunk(2, 1)
    H, scales = _scaled(g * torch.sigmoid(g) * u)
    return {"H": H, "scales": scales}


def _exact_product(s, halves):
    """sum over blocks b of d: A_scale[b] W_scale[n, b] (codes of A) . (codes of W)."""
    off = s["offsets"].tolist()
    E, N, d = s["W"].shape
    n = N // halves
    S = off[-1]
    token = s["perm"].long().div(s["c"]["k"], rounding_mode="floor") if s["perm"] is not None else None
    out = torch.zeros(S, N, dtype=torch.float64, device=s["W"].device)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        src = token[lo:hi] if token is not None else torch.arange(lo, hi, device=out.device)
        a = s["A"].view(torch.uint8)[src].view(E4M3).double() * s["As"][src].double().repeat_interleave(BLOCK, 1)[:, :d]
        ws = s["Ws"][e].double().repeat_interleave(BLOCK, 1)[:, :d].reshape(halves, _blocks(n), d)
        w = s["W"][e].double() * ws.repeat_interleave(BLOCK, 1)[:, :n].reshape(N, d)
        out[lo:hi] = torch.einsum("sd,nd->sn", a, w)
    return out


def _exact_router(s):
    """The losses as functions of the logits, and their gradient (with the gates') by automatic differentiation."""
    c = s["c"]
    T, E, k = c["T"], c["E"], c["k"]
    L = c["seq"] or T
    logits = s["logits"].double().requires_grad_(True)
    idx = s["topk_idx"].long()
    mask = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=logits.device)
    score = torch.sigmoid(logits) if c["gates"].startswith("sigmoid") else torch.softmax(logits, 1)
    p = score / score.sum(1, keepdim=True)
    edges = list(range(0, T, L))
    load, tokens, balance = [], [], logits.new_zeros(())
    for t0 in edges:
        m = mask[t0:t0 + L]
        count = torch.bincount(idx[t0:t0 + L][m].reshape(-1), minlength=E)
        n = int(m.sum())
        load.append(count)
        tokens.append(n)
        if n:
            f = count.double() * (E / (k * n))
            balance = balance + (f * (p[t0:t0 + L] * m[:, None]).sum(0) / n).sum() * (BALANCE / len(edges))
    counted = max(1, sum(tokens))
    z = Z * (torch.logsumexp(logits, 1).square() * mask).sum() / counted
    gate = score.gather(1, idx)
    if c["gates"].endswith("renorm"):
        gate = gate / gate.sum(1, keepdim=True)
    (balance + z + (gate * s["dw"].double()).sum()).backward()
    return {"loss": torch.stack([balance, z]).detach(), "load": torch.stack(load).to(torch.int32),
            "tokens": torch.tensor(tokens + [sum(tokens)], dtype=torch.int32, device=logits.device),
            "dlogits": logits.grad}
