"""The workspace's area of split reductions: what an earlier call left in it does not matter."""
import numpy as np
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fill", [0xFF, 0x7F, 0x01])
def test_the_split_area_may_hold_anything(fill):
    """A valid call takes nothing from it, and one whose offsets are no segments writes nothing by its list."""
    counts, d, N = [4501, 70, 0, 6213], 80, 4624
    S, E = sum(counts), len(counts)
    plan = binding.moe_plan(S, d, E, 1, N)
    # the last part of the workspace, 256-byte aligned: the list of at most 256 tiles, and a slot of 256 x 256 sums for each SM
    area = 32 + 256 * 40 + torch.cuda.get_device_properties(0).multi_processor_count * 256 * 256 * 4
    first = (plan.workspace_bytes - area) // 256 * 256
    assert first > 0
    g = torch.Generator(device="cuda").manual_seed(3)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    A, dY, W = ints(S, d), ints(S, N), ints(E, d, N)
    off = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device="cuda")
    bad = off.clone()
    bad[1] = S + 1
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    ends = off.tolist()
    want_a = torch.cat([dY[a:b].float() @ W[e].float().T for e, (a, b) in enumerate(zip(ends, ends[1:]))])
    want_w = torch.stack([A[a:b].float().T @ dY[a:b].float() for a, b in zip(ends, ends[1:])])
    for o, ok in ((bad, False), (off, True)):
        dA = torch.full((S, d), float("nan"), device="cuda")
        dW = torch.full((E, d, N), float("nan"), device="cuda")
        for run in (lambda: binding.moe_grouped_gemm_dgrad(plan, dY, o, W, dA, ws, st),
                    lambda: binding.moe_grouped_gemm_wgrad(plan, A, dY, o, dW, ws, st)):
            ws[first:] = fill
            st.zero_()
            run()
            assert binding.moe_read_status(st)[0] == (binding.MOE_OK if ok else binding.MOE_ERR_DEVICE)
        if ok:  # whole numbers below 2^24: every sum is exact
            assert torch.equal(dA, want_a) and torch.equal(dW, want_w)
        else:
            assert torch.isnan(dA).all() and torch.isnan(dW).all()
