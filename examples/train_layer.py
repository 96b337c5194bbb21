"""Trains one MoE layer to reproduce another's outputs: every training operator of the library in one
step, with plain gradient descent.

    python examples/train_layer.py [--steps 60] [--tokens 512] [--width 512] [--hidden 704] [--experts 8] [--top 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_token_dispatch_route_gb300 import binding  # noqa: E402
from moe_token_dispatch_route_gb300.training import MoeTrainLayer  # noqa: E402


def weights(d, F, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return torch.randn(shape, generator=g, device="cuda") * scale
    return {"W_r": normal(d, E, scale=d ** -0.5), "W1": normal(E, d, 2 * F, scale=d ** -0.5),
            "W2": normal(E, F, d, scale=F ** -0.5), "gamma": 1 + normal(d, scale=0.1), "beta": normal(d, scale=0.1)}


def train(steps, T, d, F, E, k, lr=0.1, seed=0):
    """Losses of the steps.  The master weights are fp32; the products take their bf16 rounding."""
    layer = MoeTrainLayer(T, d, F, E, k)
    low = lambda p: {n: v.bfloat16() if n.startswith("W") else v for n, v in p.items()}  # noqa: E731
    x = torch.randn(T, d, generator=torch.Generator(device="cuda").manual_seed(seed + 9), device="cuda")
    want = layer.forward(x, **low(weights(d, F, E, seed + 1))).clone()
    p = weights(d, F, E, seed + 2)
    grads = {n: torch.empty_like(v) for n, v in p.items()}
    losses = []
    for _ in range(steps):
        q = low(p)
        err = layer.forward(x, **q) - want
        losses.append((err * err).mean())
        layer.backward(err * (2.0 / T), x, q["gamma"], q["W_r"], q["W1"], q["W2"], grads)
        for n, v in p.items():
            v.add_(grads[n], alpha=-lr)
    rc, status = binding.moe_read_status(layer.bufs.status)
    if rc != 0:
        raise RuntimeError(f"device status {status}")
    return [float(v) for v in losses], layer


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, value in (("steps", 60), ("tokens", 512), ("width", 512), ("hidden", 704), ("experts", 8), ("top", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    losses, layer = train(a.steps, a.tokens, a.width, a.hidden, a.experts, a.top)
    for i in sorted({*range(0, a.steps, 10), a.steps - 1}):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"held between the passes: {layer.kept_bytes() / 2**20:.1f} MiB")
