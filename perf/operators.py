"""Cases that measure the training operators of a Mixture-of-Experts layer: layer norm and its gradient,
the SwiGLU activation with its 8-bit checkpoint and that checkpoint's use in the backward pass, the two
gradients of the per-expert grouped product, and the gradient of the gate-weighted combine.

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits; with ``own`` true it
makes the calls of this repository's package.  ``exact`` states each operator once more in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 128    # columns that share one scale of the 8-bit checkpoint
EPS = 1e-5


def listed():
    return [
        # a decode batch of 64 token rows normalised before the router: latency
        dict(name="layernorm_decode", op="layernorm", T=64, d=4096, x="bf16"),
        # a small training batch of odd size, fp32 residual stream: the gradient at latency-bound size
        dict(name="layernorm_backward_small", op="layernorm_backward", T=333, d=2064, x="f32", dy="f32"),
        # the norm before a Mixtral-shaped layer: bf16 residual stream, fp32 gradient from the combined experts
        dict(name="layernorm_backward_mixtral", op="layernorm_backward", T=8192, d=4096, x="bf16", dy="f32"),
        # activation of the fine-grained layer (F = 1408): stored in 8 bits, then used by the backward pass
        dict(name="swiglu_step_finegrained", op="swiglu_step", T=16384, k=4, F=1408, gu="bf16", dh="bf16"),
        # the backward pass alone on the Mixtral-shaped layer (F = 14336)
        dict(name="swiglu_backward_mixtral", op="swiglu_backward", T=8192, k=2, F=14336, gu="bf16", dh="bf16"),
        # the tiny layer's input gradient: latency
        dict(name="dgrad_tiny", op="dgrad", T=256, d=512, E=8, k=2, N=1024, load="none", out="f32"),
        # a decode-sized batch over 128 experts, four of them hot: the weights' bytes
        dict(name="dgrad_decode", op="dgrad", T=64, d=4096, E=128, k=8, N=1536, load="hot4", out="bf16"),
        # the Mixtral-shaped layer's input gradient: tensor-core work
        dict(name="dgrad_mixtral", op="dgrad", T=8192, d=4096, E=8, k=2, N=14336, load="none", out="bf16"),
        # weight gradient of the fine-grained layer, Zipf load, experts without rows
        dict(name="wgrad_finegrained", op="wgrad", T=16384, d=2048, E=64, k=4, N=1408, load="zipf", out="f32"),
        # weight gradient of the Mixtral-shaped layer
        dict(name="wgrad_mixtral", op="wgrad", T=8192, d=4096, E=8, k=2, N=14336, load="none", out="f32"),
        # gradient of the combine, small batch of odd size with bf16 expert outputs
        dict(name="combine_backward_small", op="combine_backward", T=333, k=4, N=1408, y="bf16", dout="bf16"),
        # gradient of the combine where 8 experts' rows of width 4096 meet in each token
        dict(name="combine_backward_wide", op="combine_backward", T=8192, k=8, N=4096, y="bf16", dout="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step=16):
    return max(lo, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    while True:
        c = _draw(rng)
        widths = [c.get("d"), c.get("N"), 2 * c.get("F", 0), c["T"], c["T"] * c.get("k", 1)]
        if 3 * 1024 not in widths:  # not a width of this package's layers
            return c


def _draw(rng):
    op = rng.choice(("layernorm", "layernorm_backward", "swiglu_step", "swiglu_backward", "dgrad", "wgrad",
                     "combine_backward"))
    ty = lambda: rng.choice(("f32", "bf16"))  # noqa: E731
    if op in ("layernorm", "layernorm_backward"):
        d = _width(rng, 64, 16384)
        c = dict(op=op, T=_log_int(rng, 1, min(32768, (1 << 27) // d)), d=d, x=ty())
        if op == "layernorm_backward":
            c["dy"] = ty()
        return c
    if op in ("swiglu_step", "swiglu_backward"):
        F, k = _width(rng, 32, 14336, 8), rng.randint(1, 8)
        return dict(op=op, T=_log_int(rng, 1, min(16384, (1 << 27) // (F * k))), k=k, F=F, gu=ty(), dh=ty())
    if op == "combine_backward":
        k, N = rng.randint(1, 8), _width(rng, 64, 8192)
        return dict(op=op, T=_log_int(rng, 1, min(16384, (1 << 28) // (k * N))), k=k, N=N, y=ty(), dout=ty())
    while True:
        E = _log_int(rng, 1, 256)
        c = dict(op=op, T=_log_int(rng, 1, 16384), d=_width(rng, 64, 8192), E=E, k=rng.randint(1, min(8, E)),
                 N=_width(rng, 64, 16384), load=rng.choice(("none", "zipf")), out=ty())
        if c["T"] * c["k"] * c["d"] * c["N"] <= 4e11 and E * c["d"] * c["N"] <= 1 << 29:
            return c


def _experts_with_rows(c):
    """Expected number of experts that receive a row (hot4: four experts hold half of the picks)."""
    E, S = c["E"], c["T"] * c["k"]
    if c["load"] == "hot4":
        return 4 + (E - 4) * (1 - math.exp(-(S - 4 * c["T"]) / (E - 4)))
    if c["load"] == "zipf":
        p = [(r + 1) ** -1.1 for r in range(E)]
        live = E - 4 if E > 4 else E  # the four least popular get no row
        live = max(live, c["k"])
        return sum(1 - math.exp(-min(S * p[r] / sum(p), c["T"])) for r in range(live))
    return E * (1 - math.exp(-S / E))


def work(c):
    size = {"f32": 4, "bf16": 2}
    T = c["T"]
    if c["op"] == "layernorm":
        return dict(bytes=T * c["d"] * (size[c["x"]] + 2) + 8 * T + 8 * c["d"], flops=7 * T * c["d"])
    if c["op"] == "layernorm_backward":  # x, dy and the residual's gradient in; dx out
        return dict(bytes=T * c["d"] * (3 * size[c["x"]] + size[c["dy"]]) + 8 * T + 12 * c["d"], flops=14 * T * c["d"])
    if c["op"] in ("swiglu_step", "swiglu_backward"):
        S, F = T * c["k"], c["F"]
        nb = -(-F // BLOCK)
        stored = 2 * F + 8 * nb
        b = S * (stored + size[c["dh"]] * F + 2 * F + 4 * F)  # codes, scales, dH in; H, dGU out
        if c["op"] == "swiglu_step":
            b += S * (2 * size[c["gu"]] * F + 2 * F + stored)
        return dict(bytes=b, flops=(30 if c["op"] == "swiglu_step" else 20) * S * F)
    if c["op"] == "combine_backward":
        S, N = T * c["k"], c["N"]
        return dict(bytes=T * N * size[c["dout"]] + S * N * (size[c["y"]] + 2) + 12 * S, flops=3 * S * N)
    S, d, N, E = T * c["k"], c["d"], c["N"], c["E"]
    if c["op"] == "dgrad":
        b = S * N * 2 + _experts_with_rows(c) * d * N * 2 + S * d * size[c["out"]]
    else:
        b = S * (d + N) * 2 + E * d * N * size[c["out"]]
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


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"c": c}
    T, op = c["T"], c["op"]

    def normal(shape, dtype, scale=1.0):
        return torch.randn(shape, generator=g, device=dev).mul_(scale).to(dtype)

    if op in ("layernorm", "layernorm_backward"):
        d = c["d"]
        x = _activations((T, d), g, dev, torch.float32) + normal((T, 1), torch.float32, 0.5)
        s["x"] = x.to(DTYPES[c["x"]])
        s["gamma"] = 1.0 + normal((d,), torch.float32, 0.1)
        s["beta"] = normal((d,), torch.float32, 0.1)
        if op == "layernorm_backward":
            x64 = s["x"].double()
            s["mean"] = x64.mean(1).float()
            s["rstd"] = (1.0 / torch.sqrt(x64.var(1, unbiased=False) + EPS)).float()
            s["dy"] = normal((T, d), DTYPES[c["dy"]], 1e-2)
            s["dres"] = normal((T, d), DTYPES[c["x"]], 1e-2)
    elif op in ("swiglu_step", "swiglu_backward"):
        S, F = T * c["k"], c["F"]
        s["gu"] = _activations((S, 2 * F), g, dev, DTYPES[c["gu"]])
        s["dh"] = normal((S, F), DTYPES[c["dh"]], 1e-2)
        if op == "swiglu_backward":  # what the forward pass left
            s["codes"], s["scales"] = _store(s["gu"])
            del s["gu"]
    elif op == "combine_backward":
        S, N = T * c["k"], c["N"]
        s["dout"] = normal((T, N), DTYPES[c["dout"]], 1e-2)
        s["Y"] = normal((S, N), DTYPES[c["y"]])
        s["topk_w"] = torch.softmax(torch.randn(T, c["k"], generator=g, device=dev), 1)
        s["dest"] = torch.randperm(S, generator=g, device=dev).to(torch.int32)
    else:
        S, d, N, E = T * c["k"], c["d"], c["N"], c["E"]
        counts = torch.bincount(_routing(c, g, dev).reshape(-1), minlength=E)
        s["counts"] = counts.tolist()  # the plain form's slices
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["dY"] = normal((S, N), torch.bfloat16, 1e-2)
        if op == "dgrad":
            s["W"] = torch.empty(E, d, N, dtype=torch.bfloat16, device=dev)
            for e in range(E):
                s["W"][e] = normal((d, N), torch.bfloat16, 1.0 / math.sqrt(d))
        else:
            s["A"] = _activations((S, d), g, dev, torch.bfloat16)
    if own:
        _handles(s, dev)
    return s


def _handles(s, dev):
    """The plan, workspace and result buffers that a program of this package keeps."""
    from moe_token_dispatch_route_gb300 import binding
    s["api"] = binding
    c, op = s["c"], s["c"]["op"]
    T = c["T"]
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
    if op in ("layernorm", "layernorm_backward"):
        d = c["d"]
        s["plan"] = binding.moe_plan(T, d, 1, 1, 256)
        if op == "layernorm":
            s["y"], s["mean"], s["rstd"] = new((T, d), torch.bfloat16), new((T,), torch.float32), new((T,), torch.float32)
        else:
            s["dx"] = new((T, d), DTYPES[c["x"]])
            s["dgamma"], s["dbeta"] = new((d,), torch.float32), new((d,), torch.float32)
            s["scratch"] = binding.backward_scratch(s["plan"])
    elif op in ("swiglu_step", "swiglu_backward"):
        S, F, k = T * c["k"], c["F"], c["k"]
        out = binding.MOE_OUT_BF16 if c["gu"] == "bf16" else binding.MOE_OUT_F32
        s["plan"] = binding.moe_plan(T, 256, max(8, k), k, 2 * F, out_dtype=out)
        if op == "swiglu_step":
            s["codes"] = new((S, 2 * F), torch.int8)
            s["scales"] = new((S, 2 * (-(-F // BLOCK))), torch.float32)
            s["H"] = new((S, F), torch.bfloat16)
        s["H_again"], s["dGU"] = new((S, F), torch.bfloat16), new((S, 2 * F), torch.bfloat16)
    elif op == "combine_backward":
        N, k = c["N"], c["k"]
        out = binding.MOE_OUT_BF16 if c["y"] == "bf16" else binding.MOE_OUT_F32
        s["plan"] = binding.moe_plan(T, 256, max(8, k), k, N, out_dtype=out)
        s["dY"], s["dw"] = new((T * k, N), torch.bfloat16), new((T, k), torch.float32)
    else:
        S, d, N, E = T * c["k"], c["d"], c["N"], c["E"]
        s["plan"] = binding.moe_plan(T, d, E, c["k"], N)
        s["workspace"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device=dev)
        s["status"] = torch.zeros(4, dtype=torch.int32, device=dev)
        s["out"] = new((S, d) if op == "dgrad" else (E, d, N), DTYPES[c["out"]])


# ---------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _PLAIN[state["c"]["op"]](state)


def _run_own(s):
    b, op, plan = s["api"], s["c"]["op"], s["plan"]
    if op == "layernorm":
        b.moe_layernorm(plan, s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "layernorm_backward":
        b.moe_layernorm_backward(plan, s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dres"], s["dx"],
                                 s["dgamma"], s["dbeta"], s["scratch"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "swiglu_step":
        b.moe_swiglu_checkpoint(plan, s["gu"], s["H"], s["codes"], s["scales"])
        b.moe_swiglu_checkpoint_backward(plan, s["dh"], s["codes"], s["scales"], s["H_again"], s["dGU"])
        return {"H": s["H"], "H_again": s["H_again"], "dGU": s["dGU"]}
    if op == "swiglu_backward":
        b.moe_swiglu_checkpoint_backward(plan, s["dh"], s["codes"], s["scales"], s["H_again"], s["dGU"])
        return {"H_again": s["H_again"], "dGU": s["dGU"]}
    if op == "combine_backward":
        b.moe_combine_backward(plan, s["dout"], s["Y"], s["topk_w"], s["dest"], s["dY"], s["dw"])
        return {"dY": s["dY"], "dtopk_w": s["dw"]}
    if op == "dgrad":
        b.moe_grouped_gemm_dgrad(plan, s["dY"], s["offsets"], s["W"], s["out"], s["workspace"], s["status"])
        return {"dA": s["out"]}
    b.moe_grouped_gemm_wgrad(plan, s["A"], s["dY"], s["offsets"], s["out"], s["workspace"], s["status"])
    return {"dW": s["out"]}


def _layernorm(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt((xc * xc).mean(1) + EPS)
    y = xc * rstd[:, None] * s["gamma"] + s["beta"]
    return {"y": y.to(torch.bfloat16), "mean": mean, "rstd": rstd}


def _layernorm_backward(s):
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dxh = dy * s["gamma"]
    dx = s["rstd"][:, None] * (dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True))
    dx = (dx + s["dres"].float()).to(s["x"].dtype)
    return {"dx": dx, "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def _blocks(v, F):
    """[S, 2F] as [S, 2, blocks, 128], padded with zeros."""
    nb = -(-F // BLOCK)
    return torch.nn.functional.pad(v.reshape(-1, 2, F), (0, nb * BLOCK - F)).reshape(-1, 2, nb, BLOCK)


def _store(gu):
    """8-bit codes and fp32 scales: scale = amax / 127 and code = nearest even of x * (127 / amax), each
    step rounded to fp32."""
    F = gu.shape[1] // 2
    b = _blocks(gu.float(), F)
    amax = b.abs().amax(-1, keepdim=True)
    live = amax > 0
    inv = torch.where(live, 127.0 / torch.where(live, amax, 1.0), 0.0)
    codes = torch.round(b * inv).to(torch.int8).reshape(-1, 2, b.shape[2] * BLOCK)[:, :, :F]
    return codes.reshape(-1, 2 * F).contiguous(), (amax / 127.0).reshape(b.shape[0], -1).contiguous()


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _swiglu_backward(s):
    F = s["codes"].shape[1] // 2
    b = _blocks(s["codes"].float(), F) * s["scales"].reshape(-1, 2, s["scales"].shape[1] // 2, 1)
    b = b.reshape(b.shape[0], 2, -1)[:, :, :F]
    g, u, dh = b[:, 0], b[:, 1], s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    act = g * sig
    dg = dh * u * (sig * (1.0 + g * (1.0 - sig)))
    return {"H_again": (act * u).to(torch.bfloat16), "dGU": torch.cat([dg, dh * act], 1).to(torch.bfloat16)}


def _swiglu_step(s):
    F = s["gu"].shape[1] // 2
    gu = s["gu"].float()
    H = (_silu(gu[:, :F]) * gu[:, F:]).to(torch.bfloat16)
    codes, scales = _store(s["gu"])
    return {"H": H, **_swiglu_backward({"codes": codes, "scales": scales, "dh": s["dh"]})}


def _combine_backward(s):
    T, k = s["topk_w"].shape
    dest = s["dest"].long()
    dout = s["dout"].float()
    dY = torch.empty(T * k, dout.shape[1], dtype=torch.bfloat16, device=dout.device)
    dY[dest] = (s["topk_w"][:, :, None] * dout[:, None, :]).to(torch.bfloat16).reshape(T * k, -1)
    dw = (s["Y"][dest].float().reshape(T, k, -1) * dout[:, None, :]).sum(-1)
    return {"dY": dY, "dtopk_w": dw}


def _dgrad(s):
    W = s["W"]
    dA = [dy.float() @ W[e].float().T for e, dy in enumerate(torch.split(s["dY"], s["counts"])) if s["counts"][e]]
    return {"dA": torch.cat(dA).to(DTYPES[s["c"]["out"]])}


def _wgrad(s):
    rows = zip(torch.split(s["A"], s["counts"]), torch.split(s["dY"], s["counts"]))
    return {"dW": torch.stack([(a.float().T @ dy.float()).to(DTYPES[s["c"]["out"]]) for a, dy in rows])}


_PLAIN = {"layernorm": _layernorm, "layernorm_backward": _layernorm_backward, "swiglu_step": _swiglu_step,
          "swiglu_backward": _swiglu_backward, "combine_backward": _combine_backward, "dgrad": _dgrad,
          "wgrad": _wgrad}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "layernorm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        return {"y": (x - mean[:, None]) * rstd[:, None] * s["gamma"].double() + s["beta"].double(), "mean": mean,
                "rstd": rstd}
    if op == "layernorm_backward":
        # dx = rstd (I - 1 1'/d - xh xh'/d) (gamma dy) + dres
        d = case["d"]
        r = s["rstd"].double()[:, None]
        xh = (s["x"].double() - s["mean"].double()[:, None]) * r
        dy = s["dy"].double()
        v = dy * s["gamma"].double()
        along = torch.einsum("td,td->t", v, xh)[:, None] / d
        dx = r * (v - v.sum(1, keepdim=True) / d - along * xh) + s["dres"].double()
        return {"dx": dx, "dgamma": torch.einsum("td,td->d", dy, xh), "dbeta": dy.sum(0)}
    if op in ("swiglu_step", "swiglu_backward"):
        F = case["F"]
        out = {}
        if op == "swiglu_step":
            gu = s["gu"].double()
            out["H"] = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
            g = _restored(gu[:, :F])
            u = _restored(gu[:, F:])
        else:
            nb = s["scales"].shape[1] // 2
            col = torch.arange(F, device=s["scales"].device) // BLOCK
            sc = s["scales"].double()
            g = s["codes"][:, :F].double() * sc[:, :nb][:, col]
            u = s["codes"][:, F:].double() * sc[:, nb:][:, col]
        sig = torch.sigmoid(g)
        dh = s["dh"].double()
        out["H_again"] = g * sig * u
        out["dGU"] = torch.cat([dh * u * (sig + g * sig * (1 - sig)), dh * g * sig], 1)
        return out
    if op == "combine_backward":
        T, k = s["topk_w"].shape
        src = torch.empty(T * k, dtype=torch.long, device=s["dest"].device)
        src[s["dest"].long()] = torch.arange(T * k, device=src.device)  # destination row -> slot
        token = src // k
        dout = s["dout"].double()
        w = s["topk_w"].double().reshape(-1)
        dw = torch.empty(T * k, dtype=torch.float64, device=src.device)
        dw[src] = torch.einsum("sn,sn->s", s["Y"].double(), dout[token])
        return {"dY": w[src][:, None] * dout[token], "dtopk_w": dw.reshape(T, k)}
    off = s["offsets"].tolist()
    if op == "dgrad":
        dA = torch.zeros(case["T"] * case["k"], case["d"], dtype=torch.float64, device=s["dY"].device)
        for e in range(case["E"]):
            dA[off[e]:off[e + 1]] = torch.einsum("sn,dn->sd", s["dY"][off[e]:off[e + 1]].double(), s["W"][e].double())
        return {"dA": dA}
    dW = torch.zeros(case["E"], case["d"], case["N"], dtype=torch.float64, device=s["dY"].device)
    for e in range(case["E"]):
        dW[e] = torch.einsum("sd,sn->dn", s["A"][off[e]:off[e + 1]].double(), s["dY"][off[e]:off[e + 1]].double())
    return {"dW": dW}


def _restored(v):
    """What the 8-bit checkpoint of one half [S, F] stands for: the fp32 roundings of its definition taken one by one."""
    F = v.shape[1]
    f32 = lambda t: t.float().double()  # noqa: E731
    out = torch.zeros_like(v)
    for c0 in range(0, F, BLOCK):
        blk = v[:, c0:c0 + BLOCK]
        amax = blk.abs().max(1, keepdim=True).values
        safe = torch.where(amax > 0, amax, torch.ones_like(amax))
        code = torch.round(f32(blk * f32(127.0 / safe)))
        out[:, c0:c0 + BLOCK] = code * f32(amax / 127.0)
    return out
