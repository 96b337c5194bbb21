"""The router's losses and the gradient of its logits against the formulas in 64 bits (differentiated automatically) and
against differences.

Tolerances.  u = 2^-24.  A score is an exponential (within 2 + 1.2 |x| units, x its argument) over a sum of E of them: with
|x| <= 16 for what matters, within (24 + E / 32 + 8) 2u of itself.  A sum over n tokens is rounded at most n / 64 + 64
times.
"""
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
I32 = torch.int32
FLAGS = {"softmax": 0, "renorm": binding.MOE_ROUTE_RENORM, "sigmoid": binding.MOE_ROUTE_SIGMOID,
         "sigmoid_renorm": binding.MOE_ROUTE_SIGMOID | binding.MOE_ROUTE_RENORM}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def setup(T, E, k, gates, masked, seq, seed=0):
    logits = torch.randn(T, E, generator=gen(seed), device=DEV) * 1.5
    idx = torch.topk(logits + torch.randn(E, generator=gen(seed + 1), device=DEV), k, 1).indices.to(I32)
    dw = torch.randn(T, k, generator=gen(seed + 2), device=DEV)
    mask = None
    if masked:
        mask = torch.rand(T, generator=gen(seed + 3), device=DEV) < 0.7
        if seq and T > seq:
            mask[:seq] = False  # a sequence without counted tokens
    plan = binding.moe_plan(T, 64, E, k, 256, route_flags=FLAGS[gates])
    return plan, logits, idx, dw, mask


def forward(plan, logits, idx, mask, seq, balance, z):
    G = binding.loss_groups(plan, seq)
    loss = torch.full((2,), float("nan"), device=DEV)
    load, tokens = torch.full((G, plan.E), -1, dtype=I32, device=DEV), torch.full((G + 1,), -1, dtype=I32, device=DEV)
    scratch = torch.full_like(binding.balance_scratch(plan, seq), 0xFF)  # NaN, -1: what it holds does not matter
    binding.moe_balance_loss(plan, logits, idx, mask, seq, balance, z, loss, load, tokens, scratch)
    return loss, load, tokens


def reference(logits, idx, dw, mask, seq, balance, z, gates):
    T, E = logits.shape
    k = idx.shape[1]
    x = logits.double().requires_grad_(True)
    m = torch.ones(T, dtype=torch.bool, device=DEV) if mask is None else mask.bool()
    score = torch.sigmoid(x) if gates.startswith("sigmoid") else torch.softmax(x, 1)
    p = score / score.sum(1, keepdim=True)
    L = seq or T
    load, tokens, bal = [], [], torch.zeros((), dtype=torch.float64, device=DEV)
    starts = range(0, T, L)
    for t0 in starts:
        mm = m[t0:t0 + L]
        c = torch.bincount(idx[t0:t0 + L][mm].long().reshape(-1), minlength=E)
        n = int(mm.sum())
        load.append(c)
        tokens.append(n)
        if n:
            bal = bal + balance / len(starts) * E / (k * n * n) * (c.double() * p[t0:t0 + L][mm].sum(0)).sum()
    N = sum(tokens)
    zl = z / max(N, 1) * torch.logsumexp(x, 1)[m].square().sum()
    total = bal + zl
    if dw is not None:
        w = score.gather(1, idx.long())
        if gates.endswith("renorm"):
            w = w / w.sum(1, keepdim=True)
        total = total + (w * dw.double()).sum()
    total.backward()
    return bal.detach(), zl.detach(), torch.stack(load).to(I32), tokens + [N], x.grad


SHAPES = [(1, 1, 1, 0), (1, 8, 2, 0), (7, 5, 5, 3), (333, 64, 4, 0), (100, 16, 2, 33), (1000, 100, 8, 128), (513, 256, 8, 512),
          (300, 1000, 6, 0), (90, 1024, 32, 1), (20000, 8, 2, 0), (5000, 32, 3, 4096)]


@pytest.mark.parametrize("T,E,k,seq", SHAPES)
@pytest.mark.parametrize("gates", list(FLAGS))
@pytest.mark.parametrize("masked", [False, True])
def test_losses_and_gradient(T, E, k, seq, gates, masked):
    plan, logits, idx, dw, mask = setup(T, E, k, gates, masked, seq)
    balance, z = 0.7, 0.3
    loss, load, tokens = forward(plan, logits, idx, mask, seq, balance, z)
    rb, rz, rload, rtokens, grad = reference(logits, idx, dw, mask, seq, balance, z, gates)
    assert torch.equal(load, rload) and tokens.tolist() == rtokens
    rel = (32 + E / 32 + T / 64 + 64 + 64) * 2 * U
    assert abs(float(loss[0]) - float(rb)) <= rel * float(rb)
    # lse is off by the units of its largest logit, and by those of the logarithm's sum
    big = float(logits.abs().max()) + 8
    assert abs(float(loss[1]) - float(rz)) <= rel * float(rz) + 0.3 * 2 * big * 64 * U * (0.0 if rtokens[-1] == 0 else 1.0) * big
    dl = torch.full_like(logits, float("nan"))
    binding.moe_router_backward(plan, logits, idx, dw, mask, seq, balance, z, load, tokens, dl)
    check_gradient(dl, grad, logits, idx, dw, load, rtokens, seq, balance, z, gates)


def check_gradient(dl, grad, logits, idx, dw, load, tokens, seq, balance, z, gates):
    """Within (score's units + a row's sums) of the magnitudes that are added up."""
    T, E = logits.shape
    k = idx.shape[1]
    x = logits.double()
    score = torch.sigmoid(x) if gates.startswith("sigmoid") else torch.softmax(x, 1)
    p = score / score.sum(1, keepdim=True)
    n = torch.tensor(tokens[:-1], dtype=torch.float64, device=DEV).clamp(min=1)
    w = (balance * E / (len(n) * k * n * n))[:, None] * load.double()
    w = w[torch.arange(T, device=DEV) // (seq or T)]
    mag = p * (w + (p * w).sum(1, keepdim=True))
    mag = mag + 2 * z / max(tokens[-1], 1) * (torch.logsumexp(x, 1).abs() + 8)[:, None] * torch.softmax(x, 1)
    if dw is not None:
        g = score.gather(1, idx.long())
        if gates.endswith("renorm"):
            g = g / g.sum(1, keepdim=True)
        picks = g * (dw.double().abs() + (g * dw.double().abs()).sum(1, keepdim=True))
        mag = mag.scatter_add(1, idx.long(), picks)
        if gates == "softmax":
            mag = mag + p * (g * dw.double().abs()).sum(1, keepdim=True)
    # The reference's own rounding: where the gradient is exactly 0 (gates of the picks alone) its 64-bit terms, each at
    # most |dw| or the losses' coefficients in magnitude and rounded to 2^-53 of itself, cancel to what is left of that.
    terms = 1 + balance * E + z * (logits.double().abs().amax(1, keepdim=True) + 8)
    terms = terms if dw is None else terms + dw.double().abs().sum(1, keepdim=True)
    bound = (32 + E / 32 + 64) * 2 * U * mag + 2.0 ** -126 + 2.0 ** -48 * terms
    torch.cuda.synchronize()
    off = (dl.double() - grad).abs()
    assert not torch.isnan(dl).any() and (off <= bound).all(), (float((off / bound).max()), int((off > bound).sum()))


@pytest.mark.parametrize("gates", list(FLAGS))
def test_parts_of_the_gradient(gates):
    """Gates alone (no losses), losses alone, one coefficient at a time."""
    T, E, k, seq = 130, 24, 3, 50
    plan, logits, idx, dw, mask = setup(T, E, k, gates, True, seq, seed=9)
    for balance, z, use in ((0.0, 0.0, True), (0.5, 0.0, False), (0.0, 0.5, False), (0.0, 0.5, True)):
        _, load, tokens = forward(plan, logits, idx, mask, seq, balance, z)
        grad = reference(logits, idx, dw if use else None, mask, seq, balance, z, gates)[4]
        dl = torch.full_like(logits, float("nan"))
        binding.moe_router_backward(plan, logits, idx if use else None, dw if use else None, mask, seq, balance, z,
                                    load if balance else None, tokens if balance or z else None, dl)
        check_gradient(dl, grad, logits, idx, dw if use else None, load, tokens.tolist(), seq, balance, z, gates)


def test_gradient_against_differences_of_the_losses():
    T, E, k, seq = 40, 12, 2, 16
    for gates in ("softmax", "sigmoid"):
        plan, logits, idx, dw, mask = setup(T, E, k, gates, True, seq, seed=5)
        step = torch.randn(T, E, generator=gen(11), device=DEV)
        _, load, tokens = forward(plan, logits, idx, mask, seq, 3.0, 0.2)
        dl = torch.empty_like(logits)
        binding.moe_router_backward(plan, logits, None, None, mask, seq, 3.0, 0.2, load, tokens, dl)
        h = 2.0 ** -6
        up = forward(plan, logits + h * step, idx, mask, seq, 3.0, 0.2)[0].double().sum()
        down = forward(plan, logits - h * step, idx, mask, seq, 3.0, 0.2)[0].double().sum()
        slope = float(up - down) / (2 * h)
        # the losses are known to 200 u of themselves (over 2 h: 4e-4 of 5), the difference's own error goes with h^2
        assert abs(slope - float((dl.double() * step.double()).sum())) <= 5e-3 * (1 + abs(slope))


def test_all_tokens_masked_and_no_tokens():
    plan, logits, idx, dw, _ = setup(50, 16, 2, "softmax", False, 0)
    mask = torch.zeros(50, dtype=torch.bool, device=DEV)
    loss, load, tokens = forward(plan, logits, idx, mask, 20, 1.0, 1.0)
    assert loss.tolist() == [0.0, 0.0] and int(load.abs().sum()) == 0 and tokens.tolist() == [0, 0, 0, 0]
    dl = torch.full_like(logits, float("nan"))
    binding.moe_router_backward(plan, logits, None, None, mask, 20, 1.0, 1.0, load, tokens, dl)
    assert (dl == 0).all()
    empty = binding.moe_plan(0, 64, 16, 2, 256)
    loss, load, tokens = forward(empty, torch.empty(0, 16, device=DEV), torch.empty(0, 2, dtype=I32, device=DEV), None, 7, 1.0, 1.0)
    assert loss.tolist() == [0.0, 0.0] and tokens.tolist() == [0, 0] and int(load.abs().sum()) == 0


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min])
@pytest.mark.parametrize("gates", ["softmax", "renorm"])
def test_masked_experts(low, gates):
    """Logits at -infinity or the type's lowest value: score and gradient 0 there, the others as without them."""
    T, E, k = 60, 40, 3
    plan, logits, idx, dw, mask = setup(T, E, k, gates, True, 0, seed=21)
    logits[:, 30:] = low
    idx = torch.topk(logits, k, 1).indices.to(I32)
    loss, load, tokens = forward(plan, logits, idx, mask, 0, 1.0, 0.1)
    dl = torch.full_like(logits, float("nan"))
    binding.moe_router_backward(plan, logits, idx, dw, mask, 0, 1.0, 0.1, load, tokens, dl)
    assert torch.isfinite(loss).all() and torch.isfinite(dl).all() and (dl[:, 30:] == 0).all()
    small = logits[:, :30].contiguous()
    rb, rz, _, rtokens, grad = reference(small, idx, dw, mask, 0, 1.0 * 40 / 30, 0.1, gates)
    assert abs(float(loss[0]) - float(rb)) <= 400 * U * float(rb)
    check_gradient(dl[:, :30], grad, small, idx, dw, load[:, :30], rtokens, 0, 1.0 * 40 / 30, 0.1, gates)


def test_far_logits():
    """Rows of logits far from zero, and picks of almost no score: the gates stay those of the picks alone."""
    T, E, k = 33, 20, 2
    plan, logits, idx, dw, _ = setup(T, E, k, "renorm", False, 0, seed=31)
    logits += 500.0
    logits[:, 0] += 300.0          # not picked, far above the picks
    idx = (1 + torch.topk(logits[:, 1:], k, 1).indices).to(I32)
    dl = torch.full_like(logits, float("nan"))
    binding.moe_router_backward(plan, logits, idx, dw, None, 0, 0.0, 0.0, None, None, dl)
    grad = reference(logits, idx, None, None, 0, 0.0, 0.0, "renorm")[4]
    x = logits.double().requires_grad_(True)
    (torch.softmax(x.gather(1, idx.long()), 1) * dw.double()).sum().backward()
    assert (grad == 0).all()
    # the differences of picks are exact to 2^-14 at 500: none of it is lost, they are the inputs' own
    assert ((dl.double() - x.grad).abs() <= 256 * U * dw.abs().sum(1, keepdim=True).double()).all()


def test_the_same_bits_on_every_run_and_in_a_graph():
    T, E, k, seq = 4000, 96, 4, 700
    plan, logits, idx, dw, mask = setup(T, E, k, "sigmoid_renorm", True, seq, seed=3)
    first = forward(plan, logits, idx, mask, seq, 1.0, 0.1)
    dl = torch.empty_like(logits)
    binding.moe_router_backward(plan, logits, idx, dw, mask, seq, 1.0, 0.1, first[1], first[2], dl)
    again = forward(plan, logits, idx, mask, seq, 1.0, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    out = [torch.zeros_like(v) for v in first]
    scratch, dl2 = binding.balance_scratch(plan, seq), torch.zeros_like(dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_balance_loss(plan, logits, idx, mask, seq, 1.0, 0.1, *out, scratch)
        binding.moe_router_backward(plan, logits, idx, dw, mask, seq, 1.0, 0.1, out[1], out[2], dl2)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, out)) and torch.equal(dl, dl2)


def test_scratch_and_coefficients_that_are_refused():
    plan, logits, idx, dw, _ = setup(5000, 64, 2, "softmax", False, 0)
    loss, load, tokens = torch.empty(2, device=DEV), torch.empty(1, 64, dtype=I32, device=DEV), torch.empty(2, dtype=I32, device=DEV)
    scratch = binding.balance_scratch(plan, 0)
    with pytest.raises(ValueError, match="scratch"):
        binding.moe_balance_loss(plan, logits, idx, None, 0, 1.0, 1.0, loss, load, tokens, scratch[:-4])
    with pytest.raises(binding.MoeError, match="WORKSPACE"):
        binding.moe_balance_loss(plan, logits, idx, None, 0, 1.0, 1.0, loss, load, tokens, None)
    for bad in (float("nan"), float("inf")):
        with pytest.raises(binding.MoeError, match="INVALID_ARG"):
            binding.moe_balance_loss(plan, logits, idx, None, 0, bad, 1.0, loss, load, tokens, scratch)
    dl = torch.empty_like(logits)
    with pytest.raises(binding.MoeError, match="INVALID_ARG"):  # a loss without its counts
        binding.moe_router_backward(plan, logits, idx, dw, None, 0, 1.0, 0.0, None, tokens, dl)
    with pytest.raises(binding.MoeError, match="INVALID_ARG"):
        binding.moe_router_backward(plan, logits, idx, dw, None, 0, 0.0, 1.0, None, None, dl)
    with pytest.raises(binding.MoeError, match="INVALID_ARG"):  # gates without their picks
        binding.moe_router_backward(plan, logits, None, dw, None, 0, 0.0, 0.0, None, None, dl)


def test_picks_outside_the_experts_are_not_counted_and_get_no_gradient():
    T, E, k = 70, 40, 3
    plan, logits, idx, dw, _ = setup(T, E, k, "sigmoid", False, 0, seed=41)
    idx[5, 1], idx[9, 2] = -1, E
    loss, load, tokens = forward(plan, logits, idx, None, 0, 1.0, 0.0)
    assert int(load.sum()) == T * k - 2
    dl = torch.full_like(logits, float("nan"))
    binding.moe_router_backward(plan, logits, idx, dw, None, 0, 0.0, 0.0, None, None, dl)
    x = logits.double().requires_grad_(True)
    ok = (idx >= 0) & (idx < E)
    (torch.sigmoid(x).gather(1, idx.clamp(0, E - 1).long()) * dw.double() * ok).sum().backward()
    assert ((dl.double() - x.grad).abs() <= 64 * U * x.grad.abs() + 2.0 ** -126).all()


@pytest.mark.parametrize("E", [128, 256, 512])
def test_logits_at_any_four_bytes(E):
    """The vectorised form is for 16-byte aligned rows; others give the same."""
    T, k = 60, 4
    plan, logits, idx, dw, mask = setup(T, E, k, "renorm", True, 25, seed=51)
    room = torch.empty(T * E + 1, device=DEV)
    room[1:] = logits.reshape(-1)
    odd = room[1:].reshape(T, E)
    results = []
    for x in (logits, odd):
        loss, load, tokens = forward(plan, x, idx, mask, 25, 1.0, 0.5)
        dl = torch.full((T * E + 1,), float("nan"), device=DEV)[1:].reshape(T, E) if x is odd else torch.full_like(x, float("nan"))
        binding.moe_router_backward(plan, x, idx, dw, mask, 25, 1.0, 0.5, load, tokens, dl)
        results.append((loss, load, tokens, dl))
    assert torch.equal(results[0][1], results[1][1]) and torch.equal(results[0][2], results[1][2])
    assert ((results[0][0] - results[1][0]).abs() <= 400 * U * results[0][0].abs()).all()
    grad = reference(logits, idx, dw, mask, 25, 1.0, 0.5, "renorm")[4]
    for _, load, tokens, dl in results:
        check_gradient(dl, grad, logits, idx, dw, load, tokens.tolist(), 25, 1.0, 0.5, "renorm")


@pytest.mark.parametrize("gates", ["sigmoid", "sigmoid_renorm"])
@pytest.mark.parametrize("E,k", [(5, 2), (8, 2), (16, 3), (30, 3), (64, 4), (256, 8), (300, 6), (1000, 6)])
@pytest.mark.parametrize("balance,z", [(0.0, 0.3), (0.7, 0.0), (0.7, 0.3)])
def test_tokens_whose_logits_are_all_far_below_zero(gates, E, k, balance, z):
    """Logistic scores that fp32 flushes to 0 (below about -87) have a sum and a share of it all the same: they are the softmax's,
    1 + e^l being 1.  Beside tokens of ordinary logits in the same warp."""
    T, seq = 61, 25
    plan, logits, idx, dw, mask = setup(T, E, k, gates, True, seq, seed=61)
    for first, shift in ((0, 100.0), (1, 60.0), (2, 500.0), (3, 20.0)):
        logits[first::5] -= shift
    dw = dw if gates == "sigmoid" else None  # (the gates of picks that are all that far below are not numbers)
    loss, load, tokens = forward(plan, logits, idx, mask, seq, balance, z)
    rb, rz, rload, rtokens, grad = reference(logits, idx, dw, mask, seq, balance, z, gates)
    assert torch.equal(load, rload) and tokens.tolist() == rtokens
    rel = (32 + E / 32 + T / 64 + 64 + 64) * 2 * U
    assert abs(float(loss[0]) - float(rb)) <= rel * float(rb)
    assert abs(float(loss[1]) - float(rz)) <= 2 * rel * float(rz)  # lse, to rel of itself, is squared
    dl = torch.full_like(logits, float("nan"))
    binding.moe_router_backward(plan, logits, None if dw is None else idx, dw, mask, seq, balance, z, load, tokens, dl)
    check_gradient(dl, grad, logits, idx, dw, load, rtokens, seq, balance, z, gates)


@pytest.mark.parametrize("T,seq", [(20, 0), (20, 5), (5000, 0), (5000, 2000)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_balance_loss_without_a_coefficient_is_zero(T, seq, bad):
    """Whatever the logits are: counted ones that are not numbers, too."""
    plan, logits, idx, dw, _ = setup(T, 16, 2, "softmax", False, seq, seed=71)
    logits[3, 4] = bad
    loss, load, tokens = forward(plan, logits, idx, None, seq, 0.0, 0.0)
    assert loss.tolist() == [0.0, 0.0] and int(load.sum()) == 2 * T and int(tokens[-1]) == T
    loss, _, _ = forward(plan, logits, idx, None, seq, 0.0, 1.0)
    assert float(loss[0]) == 0.0 and not torch.isfinite(loss[1])


@pytest.mark.parametrize("gates", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [6, 8, 16, 48, 64, 256, 1000])
@pytest.mark.parametrize("step", [0, 1])
def test_balance_gradient_of_an_even_and_a_nearly_even_load(gates, E, step):
    """p (w - sum p w) is the same for w less any constant, and what the load's common part adds cancels: it is 0 for an even
    load, and for a nearly even one known to the rounding of what differs (the scores' units and a row's sums)."""
    T, k, balance = 50, 2, 0.7
    plan, logits, idx, _, _ = setup(T, E, k, gates, False, 0, seed=81)
    load = torch.full((1, E), 10000, dtype=I32, device=DEV)
    load[0, ::2] += step
    tokens = torch.full((2,), 10000 * E // k, dtype=I32, device=DEV)
    dl = torch.full_like(logits, float("nan"))
    binding.moe_router_backward(plan, logits, None, None, None, 0, balance, 0.0, load, tokens, dl)
    if step == 0:
        assert (dl == 0).all()
        return
    x = logits.double()
    score = torch.sigmoid(x) if gates == "sigmoid" else torch.softmax(x, 1)
    p = score / score.sum(1, keepdim=True)
    n = float(tokens[0])
    w = (balance * E / (k * n * n)) * (load[0].double() - load[0].double().mean())
    grad = p * (w - (p * w).sum(1, keepdim=True)) * ((1 - score) if gates == "sigmoid" else 1)
    mag = p * (w.abs() + (p * w.abs()).sum(1, keepdim=True))
    # the mean is rounded once: a constant of 10000 u beside differences of a half, whose share is p times 1 - sum p, both
    # known to the units below
    bound = (32 + E / 32 + 64) * 2 * U * (1 + 10000 * U / 0.5) * mag + 2.0 ** -126
    torch.cuda.synchronize()
    off = (dl.double() - grad).abs()
    assert (off <= bound).all(), (float((off / bound).max()), int((off > bound).sum()))
