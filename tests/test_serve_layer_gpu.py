"""The 8-bit layer: each stage of a pass against the formula in 64 bits on what the stage before stored, passes in a captured
graph, layers that share weights.  Tolerances as in test_fp8_gpu.py."""
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding
from moe_token_dispatch_route_gb300.serving import MoeServeLayer

from .test_fp8_gpu import BF16, DEV, F32, U, check_8bit, product, product_rounds, randn, rms_ref, within

pytestmark = pytest.mark.gpu


def make(T, d, F, E, k, seed=0, **kw):
    gamma = 1 + randn((d,), seed, scale=0.1)
    W_r = randn((d, E), seed + 1, BF16, d ** -0.5)
    W1, W2 = randn((E, d, 2 * F), seed + 2, BF16, d ** -0.5), randn((E, F, d), seed + 3, BF16, F ** -0.5)
    return MoeServeLayer(T, gamma, W_r, W1, W2, k, **kw), W1, W2


@pytest.mark.parametrize("T,d,F,E,k", [(1, 64, 32, 4, 2), (7, 144, 48, 3, 3), (64, 512, 272, 16, 4), (700, 256, 400, 2, 2)])
@pytest.mark.parametrize("x_dtype,h_dtype", [(F32, BF16), (BF16, F32)])
def test_stages_of_a_pass(T, d, F, E, k, x_dtype, h_dtype):
    layer, W1, W2 = make(T, d, F, E, k)
    x, res = randn((T, d), 9, x_dtype), randn((T, d), 10, h_dtype, 3.0)
    h = res.clone()
    out = layer.forward(x, h)
    assert binding.moe_read_status(layer.status)[0] == 0
    hr, _, y = rms_ref(x, res, layer.gamma, h_dtype)
    assert torch.equal(h, hr)
    err = ((d / 64 + 64) / 2 + 8) * U * y.abs()
    within(layer.y, y, err + 2.0 ** -8 * y.abs(), "y")
    check_8bit(layer.codes, layer.scales, y, err, "rows")
    # routing is of the bf16 rows
    logits = layer.y.double() @ layer.W_r.double()
    within(layer.logits, logits, d * U * (layer.y.double().abs() @ layer.W_r.double().abs()), "logits")
    top = torch.topk(layer.logits, k, 1)
    assert torch.equal(top.values, layer.logits.gather(1, layer.topk_idx.long()))
    assert torch.equal(layer.perm[layer.dest.long()], torch.arange(T * k, device=DEV, dtype=torch.int32))
    c1, s1, c2, s2 = layer.weights
    gu, mag = product((layer.offsets, layer.perm, layer.codes, layer.scales, c1, s1), k, 2)
    g, u = gu[:, :F], gu[:, F:]
    e = product_rounds(d) * U * mag
    ref = g * torch.sigmoid(g) * u
    err = 1.1 * u.abs() * e[:, :F] + (g * torch.sigmoid(g)).abs() * e[:, F:] + e[:, :F] * e[:, F:] + (8 + 1.2 * g.abs()) * 2 * U * ref.abs()
    check_8bit(layer.H, layer.H_scales, ref, err, "H")
    Y, mag = product((layer.offsets, None, layer.H, layer.H_scales, c2, s2), k, 1)
    err = product_rounds(F) * U * mag + 2.0 ** -8 * Y.abs()
    w, at = layer.topk_w.double(), layer.dest.long().reshape(T, k)
    sums = (w[:, :, None] * Y[at]).sum(1)
    size = (w[:, :, None] * Y[at].abs()).sum(1)
    within(out, sums, (w[:, :, None] * err[at]).sum(1) + (k + 1) * 2 * U * size, "out")


def test_eight_bits_are_near_the_layer_of_whole_weights():
    """Each value of the operands is off by at most 2^-4 of itself (or 2^-10 of its block's scale), so a product of
    two is off by 2^-3 of itself: the down projection's share of the error is bounded by the terms' magnitudes."""
    T, d, F, E, k = 33, 256, 128, 4, 2
    layer, W1, W2 = make(T, d, F, E, k, seed=20)
    h = randn((T, d), 30, BF16)
    layer.forward(None, h)
    Hf = layer.H.double() * layer.H_scales.double().repeat_interleave(128, 1)[:, :F]
    off = layer.offsets.tolist()
    exact = torch.cat([Hf[off[e]:off[e + 1]] @ W2[e].double() for e in range(E)])
    # the codes' own half steps of W2, at their block's largest value
    slack = torch.cat([Hf[off[e]:off[e + 1]].abs() @ (2.0 ** -4 * W2[e].double().abs() + 2.0 ** -10 * W2[e].double().abs().max() / 448)
                       for e in range(E)])
    within(layer.Y, exact, slack * 1.001 + 2.0 ** -8 * (exact.abs() + slack), "Y")


def test_a_captured_pass_follows_its_inputs():
    T, d, F, E, k = 64, 256, 128, 16, 4
    layer, _, _ = make(T, d, F, E, k, seed=40)
    x, h = randn((T, d), 50), randn((T, d), 51, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x, h.clone())
    torch.cuda.current_stream().wait_stream(side)
    state = h.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, state)
    for seed in (60, 61):
        x.copy_(randn((T, d), seed))
        state.copy_(h)
        graph.replay()
        got, stream_state = layer.out.clone(), state.clone()
        again = h.clone()
        want = layer.forward(x, again)
        assert torch.equal(got, want) and torch.equal(stream_state, again)
    assert binding.moe_read_status(layer.status)[0] == 0


def test_layers_of_other_sizes_share_the_weights():
    d, F, E, k = 128, 64, 8, 2
    big, _, _ = make(96, d, F, E, k, seed=70)
    small = MoeServeLayer(5, None, None, None, None, 0, like=big)
    assert small.weights is big.weights and big.weight_bytes() < 1.01 * E * 3 * d * F + 4 * E * 3
    h = randn((96, d), 80, BF16)
    whole = big.forward(None, h).clone()
    assert torch.equal(small.forward(None, h[:5].contiguous()), whole[:5])


def test_two_layers_hand_the_stream_on():
    """The second layer adds the first one's sum to the stream that it normed."""
    T, d = 40, 128
    one, _, _ = make(T, d, 64, 4, 2, seed=90)
    two, _, _ = make(T, d, 64, 4, 2, seed=95)
    h = randn((T, d), 99, BF16)
    start = h.clone()
    first = one.forward(None, h)
    assert torch.equal(h, start)
    kept = first.clone()
    two.forward(first, h)
    assert torch.equal(h, (kept + start.float()).to(BF16))


def test_weights_that_do_not_fit_are_refused():
    d, F, E = 64, 32, 4
    gamma, W_r = torch.ones(d, device=DEV), randn((d, E), 1, BF16)
    W1, W2 = randn((E, d, 2 * F), 2, BF16), randn((E, F, d), 3, BF16)
    for bad in (dict(W2=W2.transpose(1, 2)), dict(W_r=W_r.float()), dict(W1=randn((E, d, 2 * F + 16), 2, BF16)), dict(gamma=gamma.half()),
                dict(selection_bias=torch.zeros(E, dtype=BF16, device=DEV))):
        a = {**dict(gamma=gamma, W_r=W_r, W1=W1, W2=W2, selection_bias=None), **bad}
        bias = a.pop("selection_bias")
        with pytest.raises(ValueError):
            MoeServeLayer(8, k=2, selection_bias=bias, **a).forward(None, randn((8, d), 4, BF16))
