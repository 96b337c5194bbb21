"""What the training calls of the binding hand to the library: a buffer that the kernels would write past its end, or
that is on another device, is refused before the call. No GPU: the library is a stand-in that records its calls, and
the tensors and the plan are on the CPU (device -1)."""
from types import SimpleNamespace

import pytest
import torch

from moe_token_dispatch_route_gb300 import binding

T, D, E, K, N = 6, 32, 4, 2, 48
S = T * K
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
WORKSPACE, SCRATCH = 4096, 1536


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(binding, "load_library", lambda *a: r)
    return r


def plan(device=-1):
    return SimpleNamespace(handle=1, device=device, T=T, d=D, E=E, N=N, S=S, workspace_bytes=WORKSPACE,
                           scratch_bytes=SCRATCH, shape=SimpleNamespace(out_dtype=binding.MOE_OUT_F32))


def buf(n, dtype=torch.uint8, device="cpu"):
    return torch.empty(n, dtype=dtype, device=device)


def dgrad(p, ws, st):
    binding.moe_grouped_gemm_dgrad(p, buf((S, N), BF16), buf(E + 1, I32), buf((E, D, N), BF16), buf((S, D), F32), ws, st, stream=0)


def wgrad(p, ws, st):
    binding.moe_grouped_gemm_wgrad(p, buf((S, D), BF16), buf((S, N), BF16), buf(E + 1, I32), buf((E, D, N), F32), ws, st,
                                   stream=0)


def norm(p, scratch, dgamma=True, dbeta=True):
    binding.moe_layernorm_backward(p, buf((T, D), F32), buf((T, D), BF16), None, buf(T, F32), buf(T, F32), None,
                                   buf((T, D), BF16), buf(D, F32) if dgamma else None, buf(D, F32) if dbeta else None,
                                   scratch, stream=0)


@pytest.mark.parametrize("call", [dgrad, wgrad])
def test_a_short_workspace_or_status_is_refused(lib, call):
    st = buf(4, I32)
    for ws in (buf(WORKSPACE - 1), buf(WORKSPACE // 4 - 1, I32), buf((WORKSPACE, 2))[:, 0], buf(0)):
        with pytest.raises(ValueError, match="workspace"):
            call(plan(), ws, st)
    for bad in (buf(3, I32), buf(8, I32)[::2], buf(15)):
        with pytest.raises(ValueError, match="dev_status"):
            call(plan(), buf(WORKSPACE), bad)
    assert lib.calls == []
    for ws in (buf(WORKSPACE), buf(WORKSPACE // 4, I32), buf(WORKSPACE + 300)):
        call(plan(), ws, st)
        args = lib.calls.pop()[1]
        assert args[-3:] == (ws.data_ptr(), st.data_ptr(), 0)


def elsewhere(n):
    return SimpleNamespace(nbytes=n, get_device=lambda: 0, device="cuda:0", is_contiguous=lambda: True, data_ptr=lambda: 256)


def test_buffers_on_another_device_are_refused(lib):
    with pytest.raises(ValueError, match="workspace is on"):
        dgrad(plan(), elsewhere(WORKSPACE), buf(4, I32))
    with pytest.raises(ValueError, match="dev_status is on"):
        wgrad(plan(), buf(WORKSPACE), elsewhere(16))
    with pytest.raises(ValueError, match="scratch is on"):
        norm(plan(), elsewhere(SCRATCH))
    assert lib.calls == []


@pytest.mark.parametrize("dgamma,dbeta", [(True, True), (True, False), (False, True)])
def test_a_short_scratch_is_refused_where_it_is_written(lib, dgamma, dbeta):
    for bad in (buf(SCRATCH - 4), buf(0), buf((SCRATCH, 2))[:, 1]):
        with pytest.raises(ValueError, match="scratch"):
            norm(plan(), bad, dgamma, dbeta)
    assert lib.calls == []
    norm(plan(), buf(SCRATCH), dgamma, dbeta)
    assert len(lib.calls) == 1


def test_what_the_library_itself_refuses_or_does_not_use_is_passed_on(lib):
    norm(plan(), None)                                  # MOE_ERR_WORKSPACE of the library
    norm(plan(), buf(8), dgamma=False, dbeta=False)     # not written: the weights' gradients are not wanted
    dgrad(plan(), None, buf(4, I32))
    wgrad(plan(), 256, 512)                             # addresses that the caller answers for
    assert [c[1][-3:] for c in lib.calls[2:]] == [(None, lib.calls[2][1][-2], 0), (256, 512, 0)]
    assert lib.calls[0][1][-2] is None
