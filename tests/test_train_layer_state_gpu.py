"""What a training layer keeps, adds to and hands out from call to call."""
import pytest
import torch

from moe_token_dispatch_route_gb300.training import MoeTrainLayer

pytestmark = pytest.mark.gpu
T, D, F, E, K = 200, 256, 208, 8, 2


def weights(seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return torch.randn(shape, generator=g, device="cuda") * scale
    return {"W_r": normal(D, E, scale=D ** -0.5).bfloat16(), "W1": normal(E, D, 2 * F, scale=D ** -0.5).bfloat16(),
            "W2": normal(E, F, D, scale=F ** -0.5).bfloat16(), "gamma": 1 + normal(D, scale=0.1), "beta": normal(D, scale=0.1)}


def batch(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, D, generator=g, device="cuda"), torch.randn(T, D, generator=g, device="cuda")


def empty_grads(p):
    return {n: torch.full(v.shape, float("nan"), device="cuda") for n, v in p.items()}


def backward(layer, dout, x, p, grads, **kw):
    return layer.backward(dout, x, p["gamma"], p["W_r"], p["W1"], p["W2"], grads, **kw)


def test_gradients_of_micro_batches_add_up():
    """All five gradients of two different batches.  Each is a sum of T or fewer fp32 terms in another order than that of
    the two alone: off by T u of the terms' magnitudes, which are below sqrt(T) of the sums' norm, 2e-4 in
    all.  (An overwritten gradient is off by half and more.)"""
    p, layer = weights(), MoeTrainLayer(T, D, F, E, K)
    alone = []
    for seed in (11, 12):
        x, dout = batch(seed)
        grads = empty_grads(p)
        layer.forward(x, **p)
        backward(layer, dout, x, p, grads)
        alone.append(grads)
    both = empty_grads(p)
    for i, seed in enumerate((11, 12)):
        x, dout = batch(seed)
        layer.forward(x, **p)
        backward(layer, dout, x, p, both, accumulate=i > 0)
    for n in p:
        want = alone[0][n] + alone[1][n]
        assert float((both[n] - want).norm()) <= 2e-4 * float(alone[0][n].norm() + alone[1][n].norm()), n


def test_a_new_layer_is_ready_for_any_stream():
    """The constructor's fills are over when it returns: a first pass on another stream waits for nothing of the stream
    that the layer was made on, and has the workspace's counters at zero."""
    p = weights()
    x, dout = batch(21)
    first = MoeTrainLayer(T, D, F, E, K)
    want = [first.forward(x, **p).clone()]
    grads = empty_grads(p)
    want += [backward(first, dout, x, p, grads)] + [grads[n] for n in sorted(p)]
    made_on, used_on = torch.cuda.Stream(), torch.cuda.Stream()
    got = empty_grads(p)
    torch.cuda.synchronize()
    with torch.cuda.stream(made_on):
        torch.cuda._sleep(200_000_000)
        layer = MoeTrainLayer(T, D, F, E, K)
        assert made_on.query()
    out = layer.forward(x, **p, stream=used_on)
    with torch.cuda.stream(used_on):
        out = out.clone()
    dx = backward(layer, dout, x, p, got, stream=used_on)
    torch.cuda.synchronize()
    for a, b in zip(want, [out, dx] + [got[n] for n in sorted(p)]):
        assert torch.equal(a, b)


def test_the_default_streams_raw_handle_is_the_default_stream():
    handle = torch.cuda.default_stream().cuda_stream
    side = torch.cuda.Stream()
    layer = MoeTrainLayer(T, D, F, E, K)
    for given, want in ((handle, handle), (side.cuda_stream, side.cuda_stream), (side, side.cuda_stream)):
        with layer._on(given):
            assert torch.cuda.current_stream().cuda_stream == want
    with torch.cuda.stream(side), layer._on(None):
        assert torch.cuda.current_stream() == side


def test_outputs_outlive_the_next_pass_and_a_backward_repeats():
    p, layer = weights(), MoeTrainLayer(T, D, F, E, K)
    (x1, dout), (x2, _) = batch(31), batch(32)
    out1 = layer.forward(x1, **p)
    kept = out1.clone()
    out2 = layer.forward(x2, **p)
    assert torch.equal(out1, kept) and not torch.equal(out1, out2)
    results = []
    for _ in range(2):
        grads = empty_grads(p)
        results.append([backward(layer, dout, x2, p, grads)] + [grads[n] for n in sorted(p)])
    assert torch.equal(out1, kept)
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_inputs_and_weights_that_require_gradients():
    """Parameters as a model holds them: the results are the same, and nothing is recorded in the layer's buffers."""
    p, layer = weights(), MoeTrainLayer(T, D, F, E, K)
    x, dout = batch(41)
    results = []
    for wanted in (False, True):
        q = {n: v.detach().clone().requires_grad_(wanted) for n, v in p.items()}
        xq = x.clone().requires_grad_(wanted)
        grads = empty_grads(p)
        for accumulate in (False, True):
            out = layer.forward(xq, **q)
            dx = backward(layer, dout, xq, q, grads, accumulate=accumulate)
        kept = [v for v in vars(layer).values() if isinstance(v, torch.Tensor)]
        assert not any(t.requires_grad for t in [out, dx, *grads.values(), *kept])
        results.append([out, dx] + [grads[n] for n in sorted(p)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_a_layer_without_tokens():
    """T = 0: nothing is read, and sums over rows are zero, or add nothing."""
    p, layer = weights(), MoeTrainLayer(0, D, F, E, K)
    x = torch.empty(0, D, device="cuda")
    assert layer.forward(x, **p).shape == (0, D)
    grads = empty_grads(p)
    assert backward(layer, x, x, p, grads).shape == (0, D)
    assert all((g == 0).all() for g in grads.values())
    for g in grads.values():
        g.fill_(1.5)
    layer.forward(x, **p)
    backward(layer, x, x, p, grads, accumulate=True)
    assert all((g == 1.5).all() for g in grads.values())


def test_a_step_in_a_graph():
    """A whole step, captured once and replayed on other inputs, gives what the calls give."""
    p, layer = weights(), MoeTrainLayer(T, D, F, E, K)
    grads = empty_grads(p)
    x, dout = batch(51)

    def step():
        out = layer.forward(x, **p)
        return [out, backward(layer, dout, x, p, grads)] + [grads[n] for n in sorted(p)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # first uses are outside the capture
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    for seed in (52, 53):
        for to, value in zip((x, dout), batch(seed)):
            to.copy_(value)
        for g in grads.values():
            g.fill_(float("nan"))
        graph.replay()
        got = [t.clone() for t in captured]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
