"""What a layer keeps of its caller's, layers of no tokens, and passes whose first call is captured."""
import os
import subprocess
import sys

import pytest
import torch

from moe_token_dispatch_route_gb300.serving import MoeServeLayer
from moe_token_dispatch_route_gb300.training import MoeTrainLayer

pytestmark = pytest.mark.gpu
DEV, BF16 = "cuda", torch.bfloat16


def weights(d, F, E):
    return (torch.ones(d, device=DEV), torch.randn(d, E, device=DEV).to(BF16), torch.randn(E, d, 2 * F, device=DEV).to(BF16),
            torch.randn(E, F, d, device=DEV).to(BF16))


def test_a_mask_that_the_caller_drops_stays_until_the_pass_has_read_it():
    T, d, F, E, k = 4096, 64, 32, 8, 2
    gamma, W_r, W1, W2 = weights(d, F, E)
    layer = MoeTrainLayer(T, d, F, E, k, norm="rms", balance=0.1)
    x, side = torch.randn(T, d, device=DEV), torch.cuda.Stream()
    layer.forward(x, gamma, None, W_r, W1, W2, stream=side)  # loads the kernels
    torch.cuda.synchronize()
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    at = mask.data_ptr()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)
    layer.forward(x, gamma, None, W_r, W1, W2, stream=side, mask=mask)
    del mask
    layer.forward(x, gamma, None, W_r, W1, W2, stream=side)  # the layer lets go of it, its first reader is still to run
    assert not side.query()
    taken = [torch.empty(T, dtype=torch.uint8, device=DEV) for _ in range(8)]
    assert at not in [t.data_ptr() for t in taken]
    torch.cuda.synchronize()


@pytest.mark.parametrize("h_dtype", [torch.float32, BF16])
def test_a_serving_layer_of_no_tokens(h_dtype):
    gamma, W_r, W1, W2 = weights(64, 32, 8)
    layer = MoeServeLayer(0, gamma, W_r, W1, W2, 2)
    h = torch.empty(0, 64, dtype=h_dtype, device=DEV)
    assert layer.forward(None, h).shape == (0, 64)
    assert layer.forward(torch.empty(0, 64, device=DEV), h).shape == (0, 64)
    torch.cuda.synchronize()
    assert layer.status.tolist() == [0, 0, 0, 0]


CAPTURE = """
import torch
from moe_token_dispatch_route_gb300.serving import MoeServeLayer
torch.manual_seed(0)
T, d, F, E, k, BF16 = {T}, 256, 128, 4, 2, torch.bfloat16
W = (torch.ones(d, device="cuda"), torch.randn(d, E, device="cuda").to(BF16) * 0.1, torch.randn(E, d, 2 * F, device="cuda").to(BF16) * 0.1,
     torch.randn(E, F, d, device="cuda").to(BF16) * 0.1)
layer = MoeServeLayer(T, *W, k)
x, h = torch.randn(T, d, device="cuda"), torch.randn(T, d, device="cuda").to(BF16)
state, graph = h.clone(), torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    layer.forward(x, state)
graph.replay()
got = layer.out.clone()
want = layer.forward(x, h.clone()).clone()
assert torch.equal(got, want) and bool(want.abs().sum() > 0)
print("same")
"""


@pytest.mark.parametrize("T", [5, 4096])  # tiles of one CTA, and of pairs
def test_the_first_pass_of_a_process_may_be_captured(T):
    r = subprocess.run([sys.executable, "-c", CAPTURE.format(T=T)], capture_output=True, text=True, timeout=200,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-1500:]
