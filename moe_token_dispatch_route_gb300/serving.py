"""One MoE layer's forward pass with weights and activations in 8 bits, on the library's calls:

    h += x,  out = combine(down(swiglu(up(dispatch(rmsnorm(h))))))

x is what the layer before hands over (an attention's output, or the layer before's `out`) and h the residual stream.  The
router sees the normed rows in bf16, the experts see them in 8 bits.
"""
from __future__ import annotations

import torch

from . import binding as b

_F32, _BF16, _I32, _E4M3 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn


class MoeServeLayer:
    """A layer for T token rows of width d: gamma fp32 [d], W_r bf16 [d, E], W1 bf16 [E, d, 2F] (gate columns, then up), W2
    bf16 [E, F, d]; d and F are multiples of 16.  The experts' weights are stored in 8 bits and not kept as they came.
    eps is 1e-5 and route_flags MOE_ROUTE_RENORM unless given; route_flags and selection_bias (fp32 [E]) as moe_route_biased takes
    them.  A program with batches of several sizes makes a layer for each and passes the first as `like`, which the others share
    everything but T with: their other arguments are None (k may be 0) or `like`'s own.
    Everything that a pass needs is allocated here, so a pass can be captured in a CUDA graph; `out` and the buffers
    belong to the stream that the passes run on: keep the layer until passes on other streams than the one that is current
    when it is made are done."""

    def __init__(self, T: int, gamma, W_r, W1, W2, k: int | None, eps: float | None = None, route_flags: int | None = None,
                 selection_bias=None, like: "MoeServeLayer | None" = None):
        if like is not None:
            other = [name for name, v in (("gamma", gamma), ("W_r", W_r), ("selection_bias", selection_bias))
                     if v is not None and v is not getattr(like, name)]
            other += [name for name, v in (("W1", W1), ("W2", W2)) if v is not None]  # like's are not kept as they came
            other += [name for name, v, none in (("k", k, (None, 0)), ("eps", eps, (None,)), ("route_flags", route_flags, (None,)))
                      if v not in none and v != getattr(like, name)]
            if other:
                raise ValueError(f"MoeServeLayer: {', '.join(other)} beside `like`, whose own are used")
            self.d, self.F, self.E, k, eps, route_flags = like.d, like.F, like.E, like.k, like.eps, like.route_flags
            gamma, W_r, selection_bias = like.gamma, like.W_r, like.selection_bias
        else:
            self.E, self.d, F2 = W1.shape
            self.F = F2 // 2
            if tuple(W2.shape) != (self.E, self.F, self.d) or tuple(W_r.shape) != (self.d, self.E) or F2 % 32:
                raise ValueError(f"MoeServeLayer: W1 {tuple(W1.shape)}, W2 {tuple(W2.shape)} and W_r {tuple(W_r.shape)} do not fit")
            eps = 1e-5 if eps is None else eps
            route_flags = b.MOE_ROUTE_RENORM if route_flags is None else route_flags
        self.T, self.k, self.eps, self.route_flags = T, k, eps, route_flags
        self.gamma, self.W_r, self.selection_bias = gamma, W_r, selection_bias
        d, F, E, S = self.d, self.F, self.E, T * k
        dev = self.device = gamma.device
        index = dev.index
        self.up = b.moe_plan(T, d, E, k, 2 * F, route_flags=route_flags, device=index)
        self.down = b.moe_plan(T, F, E, k, d, out_dtype=b.MOE_OUT_BF16, device=index)

        def new(*shape, dtype=_F32):
            return torch.empty(shape, dtype=dtype, device=dev)
        if like is not None:
            self.weights = like.weights
        else:
            # the router's call takes its weights by address alone: one of another type would be misread
            b._arg("MoeServeLayer", self.up, "W_r", W_r, d * E, b._IS_BF16)
            b._opt("MoeServeLayer", self.up, "selection_bias", selection_bias, E, b._IS_F32)
            c1, s1 = new(E, 2 * F, d, dtype=_E4M3), new(E, 2 * b.scale_blocks(F), b.scale_blocks(d))
            c2, s2 = new(E, d, F, dtype=_E4M3), new(E, b.scale_blocks(d), b.scale_blocks(F))
            b.moe_quantize_weights(self.up, W1, c1, s1, halves=2)
            b.moe_quantize_weights(self.down, W2, c2, s2)
            self.weights = (c1, s1, c2, s2)
        self.y, self.codes, self.scales = new(T, d, dtype=_BF16), new(T, d, dtype=_E4M3), new(T, b.scale_blocks(d))
        self.logits, self.topk_idx, self.topk_w = new(T, E), new(T, k, dtype=_I32), new(T, k)
        self.counts, self.offsets = new(E, dtype=_I32), new(E + 1, dtype=_I32)
        self.perm, self.dest = new(S, dtype=_I32), new(S, dtype=_I32)
        self.H, self.H_scales, self.Y = new(S, F, dtype=_E4M3), new(S, b.scale_blocks(F)), new(S, d, dtype=_BF16)
        self.out = new(T, d)
        self.up_ws = torch.zeros(self.up.workspace_bytes, dtype=torch.uint8, device=dev)
        self.down_ws = torch.zeros(self.down.workspace_bytes, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(4, dtype=_I32, device=dev)
        # the fills and the weights above are over before any stream uses them
        torch.cuda.current_stream(dev).synchronize()

    def forward(self, x, h, stream=None):
        """h (fp32 or bf16 [T, d]) += x (fp32 or bf16 [T, d]; None: nothing to add), and the experts' sum of its normed rows: `out`,
        fp32 [T, d], the layer's own, which the next pass overwrites."""
        c1, s1, c2, s2 = self.weights
        u, dn = self.up, self.down
        if x is None:
            b.moe_rmsnorm(u, h, None, self.gamma, self.eps, None, self.y, self.codes, self.scales, stream=stream)
        else:
            b.moe_rmsnorm(u, x, h, self.gamma, self.eps, h, self.y, self.codes, self.scales, stream=stream)
        b.moe_router_logits(u, self.y, self.W_r, None, self.logits, stream)
        b.moe_route_biased(u, self.logits, self.selection_bias, self.topk_idx, self.topk_w, self.counts, self.offsets,
                           self.perm, self.dest, self.up_ws, stream)
        b.moe_grouped_gemm_fp8_swiglu(u, self.codes, self.scales, self.perm, self.offsets, c1, s1, self.H, self.H_scales,
                                      self.up_ws, self.status, stream)
        b.moe_grouped_gemm_fp8(dn, self.H, self.H_scales, None, self.offsets, c2, s2, self.Y, self.down_ws, self.status, stream)
        b.moe_combine(dn, self.Y, self.topk_w, self.dest, self.out, stream)
        return self.out

    def weight_bytes(self) -> int:
        """What the experts' weights take on the device."""
        return sum(t.numel() * t.element_size() for t in self.weights)
