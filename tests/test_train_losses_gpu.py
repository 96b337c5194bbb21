"""The training layer with the RMS norm and the router's losses, against automatic differentiation of its formula in 64 bits.
Tolerance as in test_train_layer_gpu.py: 3% of each gradient's norm for what passes through bf16 and the 8-bit checkpoint."""
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding
from moe_token_dispatch_route_gb300.training import MoeTrainLayer

pytestmark = pytest.mark.gpu
REL = 3e-2
DEV = "cuda"


def weights(d, F, E, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda shape, scale: torch.randn(shape, generator=g, device=DEV) * scale  # noqa: E731
    return dict(gamma=1 + rand((d,), 0.1), W_r=rand((d, E), d ** -0.5).bfloat16(), W1=rand((E, d, 2 * F), d ** -0.5).bfloat16(),
                W2=rand((E, F, d), F ** -0.5).bfloat16())


def reference(x, p, topk_idx, F, mask, seq, balance, z, eps=1e-5):
    """(output, balance loss, z loss) in 64 bits with the given routing, differentiable."""
    T, k = topk_idx.shape
    E = p["W1"].shape[0]
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * p["gamma"]
    logits = y @ p["W_r"]
    gates = torch.softmax(logits.gather(1, topk_idx), 1)
    out = x
    for e in range(E):
        t, j = (topk_idx == e).nonzero(as_tuple=True)
        gu = y[t] @ p["W1"][e]
        h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        out = out.index_add(0, t, gates[t, j][:, None] * (h @ p["W2"][e]))
    m = torch.ones(T, dtype=torch.bool, device=DEV) if mask is None else mask
    prob = torch.softmax(logits, 1)
    starts = range(0, T, seq or T)
    bal = x.new_zeros(())
    for t0 in starts:
        mm = m[t0:t0 + (seq or T)]
        n = int(mm.sum())
        if n:
            c = torch.bincount(topk_idx[t0:t0 + (seq or T)][mm].reshape(-1), minlength=E).double()
            bal = bal + balance / len(starts) * E / (k * n * n) * (c * prob[t0:t0 + (seq or T)][mm].sum(0)).sum()
    zl = z * torch.logsumexp(logits, 1)[m].square().mean()
    return out, bal, zl


@pytest.mark.parametrize("T,d,F,E,k,seq,masked", [(200, 256, 208, 8, 2, 0, False), (129, 128, 144, 4, 1, 50, True),
                                                  (700, 272, 320, 6, 3, 128, True)])
def test_gradients_with_the_losses(T, d, F, E, k, seq, masked):
    p = weights(d, F, E, 3)
    # coefficients at which the losses' gradients of the router are as large as the gates'
    balance, z = 20.0, 5.0
    layer = MoeTrainLayer(T, d, F, E, k, norm="rms", balance=balance, z=z, seq_len=seq)
    g = torch.Generator(device=DEV).manual_seed(4)
    x, dout = torch.randn(T, d, generator=g, device=DEV) + 0.3, torch.randn(T, d, generator=g, device=DEV)
    mask = torch.rand(T, generator=g, device=DEV) < 0.6 if masked else None
    out = layer.forward(x, p["gamma"], None, p["W_r"], p["W1"], p["W2"], mask=mask)
    grads = {n: torch.full(v.shape, float("nan"), device=DEV) for n, v in p.items()}
    back = lambda acc: layer.backward(dout, x, p["gamma"], p["W_r"], p["W1"], p["W2"], grads, accumulate=acc)  # noqa: E731
    dx = back(False)
    assert binding.moe_read_status(layer.bufs.status)[0] == 0
    p64 = {n: v.double().requires_grad_() for n, v in p.items()}
    x64 = x.double().requires_grad_()
    ref, bal, zl = reference(x64, p64, layer.bufs.topk_idx.long(), F, mask, seq, balance, z)
    ((ref * dout.double()).sum() + bal + zl).backward()
    # the logits are of bf16 rows: 2^-8 of the rows' spread
    assert abs(float(layer.loss[0]) - float(bal)) <= 1e-2 * float(bal)
    assert abs(float(layer.loss[1]) - float(zl)) <= 1e-2 * float(zl)
    ref = ref.detach()
    assert float((out.double() - ref).norm()) <= 1e-2 * float((ref - x.double()).norm())
    for name, got, want in [("x", dx, x64.grad)] + [(n, grads[n], p64[n].grad) for n in p]:
        assert torch.isfinite(got).all(), name
        assert float((got.double() - want).norm()) <= REL * float(want.norm()), name
    first = {n: v.clone() for n, v in grads.items()}
    back(True)
    for n in grads:
        assert float((grads[n] - 2 * first[n]).norm()) <= 1e-5 * float(first[n].norm()), n


def test_losses_alone_leave_the_output_and_add_to_the_router():
    T, d, F, E, k = 150, 128, 112, 8, 2
    p = weights(d, F, E, 7)
    beta = torch.zeros(d, device=DEV)
    x, dout = torch.randn(T, d, device=DEV), torch.randn(T, d, device=DEV)
    results = []
    for kw in (dict(), dict(balance=1e-30, z=0.0), dict(balance=0.0, z=1.0)):
        layer = MoeTrainLayer(T, d, F, E, k, **kw)
        out = layer.forward(x, p["gamma"], beta, p["W_r"], p["W1"], p["W2"])
        grads = {n: torch.empty(v.shape, device=DEV) for n, v in {**p, "beta": beta}.items()}
        dx = layer.backward(dout, x, p["gamma"], p["W_r"], p["W1"], p["W2"], grads)
        results.append((out, dx, grads, layer))
    plain, tiny, zed = results
    assert plain[3].loss is None and plain[3].load is None
    assert torch.equal(plain[0], tiny[0]) and torch.equal(plain[0], zed[0])
    # a coefficient that adds nothing: the gates' gradient by the library's call and by PyTorch's operations
    for n in grads:
        assert float((plain[2][n] - tiny[2][n]).norm()) <= 1e-5 * float(plain[2][n].norm()), n
    assert int(tiny[3].load.sum()) == T * k
    assert float((zed[2]["W_r"] - plain[2]["W_r"]).norm()) > 0
    assert torch.equal(zed[2]["W1"], plain[2]["W1"])


def test_a_mask_that_is_refilled_before_the_backward_pass():
    """The backward pass is that of the mask which the forward pass was given."""
    T, d, F, E, k, seq = 150, 128, 112, 8, 2, 40
    p = weights(d, F, E, 7)
    g = torch.Generator(device=DEV).manual_seed(8)
    x, dout = torch.randn(T, d, generator=g, device=DEV), torch.randn(T, d, generator=g, device=DEV)
    mask = torch.rand(T, generator=g, device=DEV) < 0.6
    layer = MoeTrainLayer(T, d, F, E, k, norm="rms", balance=20.0, z=5.0, seq_len=seq)
    results = []
    for refill in (False, True):
        given = mask.clone()
        layer.forward(x, p["gamma"], None, p["W_r"], p["W1"], p["W2"], mask=given)
        if refill:
            given.logical_not_()
        grads = {n: torch.full(v.shape, float("nan"), device=DEV) for n, v in p.items()}
        dx = layer.backward(dout, x, p["gamma"], p["W_r"], p["W1"], p["W2"], grads)
        results.append((dx, grads["W_r"]))
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(*results))


def test_passes_with_and_without_a_mask_alternate():
    T, d, F, E, k = 70, 64, 32, 8, 2
    p = weights(d, F, E, 7)
    x = torch.randn(T, d, device=DEV)
    layer = MoeTrainLayer(T, d, F, E, k, norm="rms", balance=1.0, z=1.0)
    mask = torch.arange(T, device=DEV) % 3 != 0
    counts = []
    for m in (None, mask, None, mask.to(torch.uint8) * 2, ~mask):
        layer.forward(x, p["gamma"], None, p["W_r"], p["W1"], p["W2"], mask=m)
        counts.append(int(layer.tokens[-1]))
    assert counts == [T, int(mask.sum()), T, int(mask.sum()), int((~mask).sum())]


def test_a_mask_of_batches_by_tokens():
    T, d, F, E, k = 60, 64, 32, 8, 2
    p = weights(d, F, E, 7)
    x = torch.randn(T, d, device=DEV)
    layer = MoeTrainLayer(T, d, F, E, k, norm="rms", balance=1.0, z=1.0, seq_len=20)
    mask = torch.arange(T, device=DEV).reshape(3, 20) % 7 < 4
    layer.forward(x, p["gamma"], None, p["W_r"], p["W1"], p["W2"], mask=mask)
    assert layer.tokens.tolist() == [*mask.sum(1).tolist(), int(mask.sum())]


def test_kept_bytes_count_what_the_losses_keep():
    T, d, F, E, k, seq = 70, 64, 32, 8, 2, 20
    plain, losses = (MoeTrainLayer(T, d, F, E, k, norm="rms", **kw) for kw in (dict(), dict(balance=1.0, seq_len=seq)))
    # logits, picks and tokens of four sequences, a mask
    assert losses.kept_bytes() - plain.kept_bytes() == 4 * T * E + 4 * 4 * E + 4 * 5 + T


def test_arguments_of_the_layer():
    with pytest.raises(ValueError):
        MoeTrainLayer(8, 64, 32, 4, 2, norm="batch")
    with pytest.raises(ValueError):
        MoeTrainLayer(8, 64, 32, 4, 2, balance=1.0, seq_len=-1)
    layer = MoeTrainLayer(8, 64, 32, 4, 2, norm="rms")
    p = weights(64, 32, 4, 1)
    with pytest.raises(ValueError, match="beta"):
        layer.forward(torch.randn(8, 64, device=DEV), p["gamma"], torch.zeros(64, device=DEV), p["W_r"], p["W1"], p["W2"])
