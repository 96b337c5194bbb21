"""One MoE layer, forward and backward, on the library's calls:

    out = x + combine(down(swiglu(up(dispatch(layernorm(x))))))

with Mixtral-style gates (softmax over the k chosen logits).  Between the two passes it keeps the
dispatched rows, the up projection's outputs in 8 bits, the experts' outputs and the routing; H is
computed again from the 8-bit values.  The router's two gradient products ([T, d] by [d, E]) and the
gates' softmax gradient over k values are PyTorch's.  Nothing is recorded for automatic differentiation: inputs
and weights may require gradients, results do not.
"""
from __future__ import annotations

import torch

from . import binding as b

_F32, _BF16 = torch.float32, torch.bfloat16


class MoeTrainLayer:
    """Plans and device buffers of a layer of T tokens of width d, E experts of hidden width F, k
    experts a token; d and F are multiples of 16.  x: fp32 [T, d].  Weights: W_r bf16 [d, E], W1 bf16
    [E, d, 2F] (gate columns, then up), W2 bf16 [E, F, d], gamma and beta fp32 [d]; their gradients
    are fp32.  `stream`: a torch stream or a raw handle; None is the current one; results belong to it.
    The buffers belong to the stream that is current when the layer is made: keep the layer until its
    passes on other streams are done."""

    def __init__(self, T: int, d: int, F: int, E: int, k: int, eps: float = 1e-5, device: int = 0):
        self.T, self.d, self.F, self.E, self.k, self.eps = T, d, F, E, k, eps
        dev = self.device = torch.device("cuda", device)
        S = T * k
        self.up = b.moe_plan(T, d, E, k, 2 * F, route_flags=b.MOE_ROUTE_RENORM, out_dtype=b.MOE_OUT_BF16, device=device)
        self.down = b.moe_plan(T, F, E, k, d, out_dtype=b.MOE_OUT_BF16, device=device)
        self.bufs = b.MoeBuffers(self.up, dev)             # routing, dispatched rows, GU, workspace, status
        self.down_ws = torch.zeros(self.down.workspace_bytes, dtype=torch.uint8, device=dev)
        self.scratch = b.backward_scratch(self.up)

        def new(*shape, dtype=_BF16):
            return torch.empty(shape, dtype=dtype, device=dev)
        # kept from the forward pass
        self.y, self.mean, self.rstd = new(T, d), new(T, dtype=_F32), new(T, dtype=_F32)
        self.codes = new(S, 2 * F, dtype=torch.int8)
        self.scales = new(S, 2 * b.checkpoint_blocks(F), dtype=_F32)
        self.Y = new(S, d)
        # passing through
        self.logits, self.out = new(T, E, dtype=_F32), new(T, d, dtype=_F32)
        self.H, self.dH, self.dY, self.dA = new(S, F), new(S, F), new(S, d), new(S, d)
        self.dw, self.dy = new(T, k, dtype=_F32), new(T, d, dtype=_F32)
        self.ones = torch.ones(T, k, dtype=_F32, device=dev)
        # the fills above, and what the memory was used for before, are over before any stream uses it
        torch.cuda.current_stream(dev).synchronize()

    def _on(self, stream):
        """Makes `stream` the current one, for the library's calls and for PyTorch's."""
        if isinstance(stream, int):  # (an ExternalStream of handle 0 is a new stream, not the default one)
            stream = torch.cuda.ExternalStream(stream, self.device) if stream else torch.cuda.default_stream(self.device)
        return torch.cuda.stream(stream)

    def forward(self, x, gamma, beta, W_r, W1, W2, stream=None):
        """The layer's output, a tensor of its own.  The layer keeps one pass: a second forward replaces what the
        first one's backward would need."""
        with torch.no_grad(), self._on(stream):
            return self._forward(x, gamma, beta, W_r, W1, W2)

    def _forward(self, x, gamma, beta, W_r, W1, W2):
        u, r = self.up, self.bufs
        # the forward calls take the weights by address alone: one of another type or size would be misread
        for name, w, n in (("W_r", W_r, self.d * self.E), ("W1", W1, self.E * self.d * 2 * self.F),
                           ("W2", W2, self.E * self.F * self.d)):
            b._arg("MoeTrainLayer.forward", u, name, w, n, b._IS_BF16)
        b.moe_layernorm(u, x, gamma, beta, self.eps, self.y, self.mean, self.rstd)
        b.moe_router_logits(u, self.y, W_r, None, self.logits)
        b.route(u, self.logits, r)
        b.dispatch_gemm(u, self.y, W1, r)                                          # GU in r.Y
        b.moe_swiglu_checkpoint(u, r.Y, self.H, self.codes, self.scales)
        b.moe_grouped_gemm(self.down, self.H, r.offsets, W2, self.Y, self.down_ws, r.status)
        b.moe_combine(self.down, self.Y, r.topk_w, r.dest, self.out)
        return torch.add(self.out, x)

    def backward(self, dout, x, gamma, W_r, W1, W2, grads: dict, accumulate: bool = False, stream=None):
        """The gradients of the latest forward pass (which may be taken more than once).  x and the weights are that pass's,
        dout fp32 [T, d].  Writes grads["W1"], ["W2"], ["W_r"], ["gamma"] and ["beta"], fp32, or
        (accumulate) adds to all of them, and returns the gradient of x."""
        with torch.no_grad(), self._on(stream):
            return self._backward(dout, x, gamma, W_r, W1, W2, grads, accumulate)

    def _backward(self, dout, x, gamma, W_r, W1, W2, grads, accumulate):
        u, dn, r = self.up, self.down, self.bufs
        b.moe_combine_backward(dn, dout, self.Y, r.topk_w, r.dest, self.dY, self.dw)
        b.moe_grouped_gemm_dgrad(dn, self.dY, r.offsets, W2, self.dH, self.down_ws, r.status)
        dGU = r.Y                                                                  # GU's buffer: its values are in the codes
        b.moe_swiglu_checkpoint_backward(u, self.dH, self.codes, self.scales, self.H, dGU)
        b.moe_grouped_gemm_wgrad(dn, self.H, self.dY, r.offsets, grads["W2"], self.down_ws, r.status, accumulate)
        b.moe_grouped_gemm_wgrad(u, r.recv[0][:u.S], dGU, r.offsets, grads["W1"], r.workspace, r.status, accumulate)
        b.moe_grouped_gemm_dgrad(u, dGU, r.offsets, W1, self.dA, r.workspace, r.status)
        b.moe_combine(dn, self.dA, self.ones, r.dest, self.dy)                     # the dispatch's gradient
        # the gates: softmax over the chosen logits
        w = r.topk_w
        dlogits = torch.zeros_like(self.logits).scatter_(
            1, r.topk_idx.long(), w * (self.dw - (w * self.dw).sum(1, keepdim=True)))
        if accumulate:
            grads["W_r"].addmm_(self.y.float().T, dlogits)
        else:
            torch.mm(self.y.float().T, dlogits, out=grads["W_r"])
        self.dy.addmm_(dlogits, W_r.float().T)
        dx = torch.empty_like(x)
        dgamma, dbeta = grads["gamma"], grads["beta"]
        if accumulate:  # the norm's gradient is written, so it goes through buffers of its own
            dgamma, dbeta = torch.empty_like(dgamma), torch.empty_like(dbeta)
        b.moe_layernorm_backward(u, self.dy, x, gamma, self.mean, self.rstd, dout, dx, dgamma, dbeta, self.scratch)
        if accumulate:
            grads["gamma"].add_(dgamma)
            grads["beta"].add_(dbeta)
        return dx

    def kept_bytes(self) -> int:
        """What the layer holds between its forward and backward pass."""
        r = self.bufs
        kept = [self.y, self.mean, self.rstd, self.codes, self.scales, self.Y, r.recv[0], r.topk_idx, r.topk_w,
                r.offsets, r.perm, r.dest]
        return sum(t.numel() * t.element_size() for t in kept)
