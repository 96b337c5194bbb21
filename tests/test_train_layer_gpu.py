"""The training operators together: a layer's outputs and gradients against automatic
differentiation of its formula in 64 bits, and a few steps of training.

Tolerance.  Relative to each gradient's norm: a value of the 8-bit checkpoint is off by at most
half of amax / 127 of its block of 128, 0.6% (rms) of values of normal spread; H, dH, dGU, Y, dY and the
dispatched rows are each rounded to bf16 (0.2% rms).  A gradient passes through at most six of these,
and the checkpoint enters it at most twice: 3% bounds it."""
import importlib.util
import os

import pytest
import torch

from moe_token_dispatch_route_gb300 import binding
from moe_token_dispatch_route_gb300.training import MoeTrainLayer

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
REL = 3e-2


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(x, p, topk_idx, F, eps=1e-5):
    """The layer in 64 bits with the given routing, differentiable."""
    mean = x.mean(1, keepdim=True)
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps) * p["gamma"] + p["beta"]
    gates = torch.softmax((y @ p["W_r"]).gather(1, topk_idx), 1)
    out = x
    for e in range(p["W1"].shape[0]):
        t, j = (topk_idx == e).nonzero(as_tuple=True)
        gu = y[t] @ p["W1"][e]
        h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        out = out.index_add(0, t, gates[t, j][:, None] * (h @ p["W2"][e]))
    return out


@pytest.mark.parametrize("T,d,F,E,k", [(200, 256, 208, 8, 2), (129, 128, 144, 4, 1), (700, 272, 320, 6, 3)])
def test_gradients_of_a_layer(example, T, d, F, E, k):
    p = {n: v.bfloat16() if n.startswith("W") else v for n, v in example.weights(d, F, E, 3).items()}
    layer = MoeTrainLayer(T, d, F, E, k)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(T, d, generator=g, device="cuda") + 0.3
    dout = torch.randn(T, d, generator=g, device="cuda")
    out = layer.forward(x, **p).clone()
    grads = {n: torch.full(v.shape, float("nan"), device="cuda") for n, v in p.items()}
    dx = layer.backward(dout, x, p["gamma"], p["W_r"], p["W1"], p["W2"], grads)
    assert binding.moe_read_status(layer.bufs.status)[0] == 0
    p64 = {n: v.double().requires_grad_() for n, v in p.items()}
    x64 = x.double().requires_grad_()
    ref = reference(x64, p64, layer.bufs.topk_idx.long(), F)
    ref.backward(dout.double())
    ref = ref.detach()
    assert float((out.double() - ref).norm()) <= 1e-2 * float((ref - x.double()).norm())
    for name, got, want in [("x", dx, x64.grad)] + [(n, grads[n], p64[n].grad) for n in p]:
        assert torch.isfinite(got).all(), name
        assert float((got.double() - want).norm()) <= REL * float(want.norm()), name
    # accumulation: the same gradients once more on top
    first = {n: v.clone() for n, v in grads.items()}
    layer.forward(x, **p)
    layer.backward(dout, x, p["gamma"], p["W_r"], p["W1"], p["W2"], grads, accumulate=True)
    torch.cuda.synchronize()
    for n in ("W1", "W2"):
        assert float((grads[n] - 2 * first[n]).norm()) <= 1e-5 * float(first[n].norm())


def test_training_lowers_the_loss(example):
    losses, layer = example.train(25, 256, 128, 208, 8, 2)
    assert losses[-1] < 0.7 * losses[0], losses
    # between the passes the up projection's outputs take 1 byte a value and 8 bytes a block pair
    S, F = 512, 208
    assert layer.codes.numel() + layer.scales.numel() * 4 == S * (2 * F + 2 * 2 * 4)


@pytest.mark.parametrize("raw", [False, True])
def test_a_layer_on_another_stream(example, raw):
    """The pass waits behind what its stream has to do, PyTorch's operations of it included."""
    T, d, F, E, k = 200, 256, 208, 8, 2
    p = {n: v.bfloat16() if n.startswith("W") else v for n, v in example.weights(d, F, E, 3).items()}
    x, dout = torch.randn(T, d, device="cuda"), torch.randn(T, d, device="cuda")
    results = []
    side = torch.cuda.Stream()
    for s in (None, side):
        layer = MoeTrainLayer(T, d, F, E, k)
        grads = {n: torch.full(v.shape, float("nan"), device="cuda") for n, v in p.items()}
        torch.cuda.synchronize()
        if s is not None:
            with torch.cuda.stream(s):
                torch.cuda._sleep(20_000_000)
        handle = s.cuda_stream if raw and s is not None else s
        out = layer.forward(x, **p, stream=handle)
        with torch.cuda.stream(s):
            out = out.clone()
            if s is not None:
                torch.cuda._sleep(20_000_000)
        dx = layer.backward(dout, x, p["gamma"], p["W_r"], p["W1"], p["W2"], grads, stream=handle)
        torch.cuda.synchronize()
        results.append([out, dx] + [grads[n] for n in sorted(grads)])
    for a, b in zip(*results):
        assert torch.equal(a, b)
