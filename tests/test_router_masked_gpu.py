"""Padding may hold anything: logits of masked tokens that are not numbers, infinite, or -infinity throughout reach neither
the losses nor the gradient. Nothing is rounded differently by their being there, so equality is to the bit."""
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding as b

pytestmark = pytest.mark.gpu
FLAGS = {"softmax": 0, "renorm": b.MOE_ROUTE_RENORM, "sigmoid": b.MOE_ROUTE_SIGMOID,
         "sigmoid_renorm": b.MOE_ROUTE_SIGMOID | b.MOE_ROUTE_RENORM}
BAD = [float("nan"), float("inf"), float("-inf"), torch.finfo(torch.float32).min]


def losses(plan, logits, idx, mask, dw, seq, balance, z):
    T, E = logits.shape
    groups = b.loss_groups(plan, seq)
    loss, load = torch.empty(2, device="cuda"), torch.empty(groups, E, dtype=torch.int32, device="cuda")
    tokens, d = torch.empty(groups + 1, dtype=torch.int32, device="cuda"), torch.empty(T, E, device="cuda")
    b.moe_balance_loss(plan, logits, idx, mask, seq, balance, z, loss, load, tokens, b.balance_scratch(plan, seq))
    b.moe_router_backward(plan, logits, idx, dw, mask, seq, balance, z, load, tokens, d)
    torch.cuda.synchronize()
    return loss, load, tokens, d


@pytest.mark.parametrize("gates", list(FLAGS))
@pytest.mark.parametrize("E,k", [(8, 2), (13, 3), (64, 4), (256, 8)])
@pytest.mark.parametrize("balance,z", [(0.01, 1e-3), (0.01, 0.0), (0.0, 1e-3)])
def test_masked_logits_that_are_not_numbers(gates, E, k, balance, z):
    T, seq = 75, 25
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(T, E, device="cuda", generator=g)
    idx = logits.topk(k, 1).indices.to(torch.int32)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    padding = torch.arange(2, T, 7, device="cuda")
    mask[padding] = 0
    mask[50:] = 0  # a whole sequence
    dirty = logits.clone()
    for i, t in enumerate((mask == 0).nonzero().flatten().tolist()):
        dirty[t] = BAD[i % len(BAD)]
        if i % 3 == 0:
            dirty[t, 1:] = logits[t, 1:]  # one expert alone
    plan = b.moe_plan(T, 16, E, k, 16, route_flags=FLAGS[gates])
    dw = torch.randn(T, k, device="cuda", generator=g)
    live = mask.bool()
    for gates_too in (None, dw):
        want = losses(plan, logits, idx, mask, gates_too, seq, balance, z)
        got = losses(plan, dirty, idx, mask, gates_too, seq, balance, z)
        for a, c in zip(got[:3], want[:3]):
            assert torch.equal(a, c)
        assert torch.equal(got[3][live], want[3][live])
        if gates_too is None:
            assert torch.equal(got[3][~live], torch.zeros_like(got[3][~live]))
        elif gates != "softmax":  # gates of the picks alone: experts that were not chosen get nothing
            rest = torch.ones(T, E, dtype=torch.bool, device="cuda").scatter_(1, idx.long(), False)[~live]
            assert torch.equal(got[3][~live][rest], torch.zeros_like(got[3][~live][rest]))
