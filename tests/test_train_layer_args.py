"""The training layer hands no weight to the library that it would misread. No GPU: the plans are stand-ins on the
CPU (device -1), and a call that gets through is recorded."""
from types import SimpleNamespace

import pytest
import torch

from moe_token_dispatch_route_gb300 import training
from moe_token_dispatch_route_gb300.training import MoeTrainLayer

T, D, F, E, K = 6, 32, 48, 4, 2
BF16 = torch.bfloat16


@pytest.fixture
def layer(monkeypatch):
    calls = []
    for name in ("moe_layernorm", "moe_router_logits", "route", "dispatch_gemm", "moe_swiglu_checkpoint", "moe_grouped_gemm",
                 "moe_combine"):
        monkeypatch.setattr(training.b, name, lambda *a, _n=name, **kw: calls.append(_n))
    v = object.__new__(MoeTrainLayer)
    v.T, v.d, v.F, v.E, v.k, v.eps = T, D, F, E, K, 1e-5
    v.up = v.down = SimpleNamespace(device=-1)
    v.bufs = SimpleNamespace(Y=None, offsets=None, status=None, topk_w=None, dest=None)
    for name in ("y", "mean", "rstd", "logits", "H", "codes", "scales", "Y", "down_ws"):
        setattr(v, name, None)
    v.out = torch.zeros(T, D)
    v.calls = calls
    return v


def weights():
    return {"W_r": torch.zeros(D, E, dtype=BF16), "W1": torch.zeros(E, D, 2 * F, dtype=BF16),
            "W2": torch.zeros(E, F, D, dtype=BF16)}


def run(layer, **w):
    return layer._forward(torch.ones(T, D), torch.ones(D), torch.zeros(D), w["W_r"], w["W1"], w["W2"])


@pytest.mark.parametrize("name", ["W_r", "W1", "W2"])
def test_a_weight_that_would_be_misread_is_refused(layer, name):
    w = weights()[name]
    for bad, word in ((w.float(), "float32"), (w[..., :-16] if name != "W_r" else w[:-1], "elements"), (None, "missing"),
                      (w.transpose(-1, -2).contiguous().transpose(-1, -2), "strided")):
        with pytest.raises(ValueError, match=f"{name} .*{word}"):
            run(layer, **{**weights(), name: bad})
    assert layer.calls == []


def test_the_weights_that_a_layer_takes(layer):
    assert torch.equal(run(layer, **weights()), torch.ones(T, D)) and len(layer.calls) == 7


def test_a_mask_is_looked_at_where_there_are_no_losses_too(layer):
    x, w = torch.ones(T, D), weights()
    args = (x, torch.ones(D), torch.zeros(D), w["W_r"], w["W1"], w["W2"])
    for bad, word in ((torch.ones(T - 1, dtype=torch.bool), "elements"), (torch.ones(T), "float32")):
        with pytest.raises(ValueError, match=f"mask .*{word}"):
            layer._forward(*args, bad)
    assert layer.calls == []
    assert torch.equal(layer._forward(*args, torch.ones(T, dtype=torch.bool)), x)  # and counts for nothing
