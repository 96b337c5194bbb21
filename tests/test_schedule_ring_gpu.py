"""The forward kernels' schedule rings when every role runs as far ahead as the ring lets it.

Tiles of one k-block and wide outputs: an epilogue warp takes its next tile while its stores of
the one before are still queued. Whole numbers: each sum is exact, so a tile that is missed, done twice or done
with another's rows shows; outputs are poisoned before each launch.
"""
import pytest
import torch

from moe_token_dispatch_route_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["dispatch", "grouped", "gather"])
@pytest.mark.parametrize("tile_m,out_dtype", [(128, binding.MOE_OUT_F32), (256, binding.MOE_OUT_F32),
                                              (256, binding.MOE_OUT_BF16)])
def test_every_tile_is_done_once_in_many_short_launches(tile_m, out_dtype, mode):
    T, d, E, k, N, launches = 1100, 64, 40, 2, 2064, 250
    plan = binding.moe_plan(T, d, E, k, N, tile_m=tile_m, out_dtype=out_dtype)
    assert plan.info["tile_m"] == tile_m
    bufs = binding.MoeBuffers(plan, "cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn(T, E, generator=g, device="cuda")
    x = (torch.arange(T, device="cuda") % 3 + 1).to(torch.bfloat16)[:, None].expand(T, d).contiguous()
    scale = 2.0 ** (torch.arange(E, device="cuda") % 4)  # an expert's rows with another's weights show too
    W = scale.to(torch.bfloat16)[:, None, None].expand(E, d, N).contiguous()
    binding.route(plan, logits, bufs)
    rows = x[(bufs.perm // k).long()].contiguous()
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), bufs.counts.long())
    want = (rows[:, :1].float() * d * scale[e][:, None]).expand(T * k, N).to(bufs.Y.dtype)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(launches):
        bufs.Y.fill_(float("nan"))
        if mode == "dispatch":
            binding.dispatch_gemm(plan, x, W, bufs)
        elif mode == "grouped":
            binding.moe_grouped_gemm(plan, rows, bufs.offsets, W, bufs.Y, bufs.workspace, bufs.status)
        else:
            binding.gather_gemm(plan, x, W, bufs)
        wrong += (bufs.Y != want).sum()
    rc, status = binding.moe_read_status(bufs.status)
    assert rc == 0, status
    assert int(wrong) == 0
