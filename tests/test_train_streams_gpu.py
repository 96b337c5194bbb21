"""The training calls on the legacy default stream, which waits for every blocking stream and is waited for by them."""
import ctypes

import pytest
import torch

from moe_token_dispatch_route_gb300 import binding

pytestmark = pytest.mark.gpu


def blocking_stream():
    """A stream of default flags (PyTorch's own do not wait for the default stream)."""
    rt = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    handle = ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(handle)) == 0
    return handle.value


def test_the_default_stream_waits_for_blocking_streams_and_they_for_it():
    T, d = 512, 1040
    plan = binding.moe_plan(T, d, 1, 1, 256)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    other = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    scratch = binding.backward_scratch(plan)

    def buffers():
        nan = lambda *s, dt=torch.float32: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
        return [nan(T, d, dt=torch.bfloat16), nan(T), nan(T), nan(T, d, dt=torch.bfloat16), nan(d), nan(d)]

    def run(x, out, stream):
        y, mean, rstd, dx, dg, db = out
        binding.moe_layernorm(plan, x, None, None, 1e-5, y, mean, rstd, stream)
        binding.moe_layernorm_backward(plan, y, x, None, mean, rstd, None, dx, dg, db, scratch, stream)

    want, warm = buffers(), buffers()
    run(x, want, 0)
    torch.cuda.synchronize()
    raw = blocking_stream()
    b = torch.cuda.ExternalStream(raw)
    late, out, copy = other.clone(), buffers(), buffers()
    torch.cuda.synchronize()
    with torch.cuda.stream(b):
        torch.cuda._sleep(50_000_000)
        late.copy_(x)
    run(other, warm, 0)   # a kernel before, whose end the next may overlap
    run(late, out, 0)
    with torch.cuda.stream(b):
        for c, o in zip(copy, out):
            c.copy_(o)
    torch.cuda.synchronize()
    for got in (out, copy):
        for a, w in zip(got, want):
            assert torch.equal(a, w)
    # the other way round: the calls on the blocking stream, their input late on the default one
    late.copy_(other)
    out = buffers()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    late.copy_(x)
    run(late, out, raw)
    torch.cuda.synchronize()
    for a, w in zip(out, want):
        assert torch.equal(a, w)
