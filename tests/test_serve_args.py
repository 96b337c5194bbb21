"""What the 8-bit forward calls and the router's losses refuse, without a GPU: the C ABI with missing plans, and the
binding with tensors the kernels would misread or write past (the library is a stand-in that records its calls, the
tensors and the plan are on the CPU, device -1)."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from moe_token_dispatch_route_gb300 import binding

NAMES = ("moe_rmsnorm", "moe_rmsnorm_backward", "moe_quantize_weights", "moe_grouped_gemm_fp8",
         "moe_grouped_gemm_fp8_swiglu", "moe_balance_scratch", "moe_balance_loss", "moe_router_backward")
T, D, E, K, N = 6, 144, 4, 2, 288
S = T * K
F32, BF16, I32, E4M3 = torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn
WORKSPACE, SCRATCH = 4096, 1536


@pytest.fixture(scope="module")
def real():
    from moe_token_dispatch_route_gb300 import build
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("name", NAMES)
def test_a_missing_plan_is_refused(real, name):
    fn = getattr(real, name)
    zero = {ctypes.c_int32: 0, ctypes.c_float: 1e-5}
    assert fn(*[zero.get(t) for t in fn.argtypes]) == binding.MOE_ERR_INVALID_ARG


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
    return SimpleNamespace(handle=1, device=device, T=T, d=D, E=E, N=N, S=S, workspace_bytes=WORKSPACE, scratch_bytes=SCRATCH,
                           shape=SimpleNamespace(out_dtype=binding.MOE_OUT_F32))


def buf(n, dtype=F32):
    return torch.empty(n, dtype=dtype)


def norm(**kw):
    a = dict(x=buf((T, D)), res=buf((T, D), BF16), gamma=buf(D), eps=1e-5, h=buf((T, D), BF16), y=buf((T, D), BF16),
             codes=buf((T, D), E4M3), scales=buf((T, 2)), rstd=buf(T), stream=0)
    binding.moe_rmsnorm(plan(), **{**a, **kw})


def norm_backward(**kw):
    a = dict(dy=buf((T, D)), h=buf((T, D), BF16), gamma=buf(D), rstd=buf(T), dres=buf((T, D), BF16), dx=buf((T, D), BF16),
             dgamma=buf(D), scratch=buf(SCRATCH, torch.uint8), stream=0)
    binding.moe_rmsnorm_backward(plan(), **{**a, **kw})


def weights(**kw):
    a = dict(W=buf((E, D, N), BF16), codes=buf((E, N, D), E4M3), scales=buf((E, 3, 2)), halves=1, stream=0)
    binding.moe_quantize_weights(plan(), **{**a, **kw})


def product(**kw):
    a = dict(A=buf((S, D), E4M3), A_scales=buf((S, 2)), perm=None, offsets=buf(E + 1, I32), W=buf((E, N, D), E4M3),
             W_scales=buf((E, 3, 2)), Y=buf((S, N)), workspace=buf(WORKSPACE, torch.uint8), dev_status=buf(4, I32), stream=0)
    binding.moe_grouped_gemm_fp8(plan(), **{**a, **kw})


def swiglu(**kw):
    a = dict(A=buf((T, D), E4M3), A_scales=buf((T, 2)), perm=buf(S, I32), offsets=buf(E + 1, I32), W1=buf((E, N, D), E4M3),
             W1_scales=buf((E, 4, 2)), H=buf((S, N // 2), E4M3), H_scales=buf((S, 2)), workspace=buf(WORKSPACE, torch.uint8),
             dev_status=buf(4, I32), stream=0)
    binding.moe_grouped_gemm_fp8_swiglu(plan(), **{**a, **kw})


def losses(**kw):
    a = dict(logits=buf((T, E)), topk_idx=buf((T, K), I32), mask=buf(T, torch.bool), seq_len=4, balance=1.0, z=1.0, loss=buf(2),
             load=buf((2, E), I32), tokens=buf(3, I32), scratch=buf(256, torch.uint8), stream=0)
    binding.moe_balance_loss(plan(), **{**a, **kw})


def losses_backward(**kw):
    a = dict(logits=buf((T, E)), topk_idx=buf((T, K), I32), dtopk_w=buf((T, K)), mask=None, seq_len=0, balance=1.0, z=1.0,
             load=buf((1, E), I32), tokens=buf(2, I32), dlogits=buf((T, E)), stream=0)
    binding.moe_router_backward(plan(), **{**a, **kw})


CALLS = {norm: "moe_rmsnorm", norm_backward: "moe_rmsnorm_backward", weights: "moe_quantize_weights",
         product: "moe_grouped_gemm_fp8", swiglu: "moe_grouped_gemm_fp8_swiglu", losses: "moe_balance_loss",
         losses_backward: "moe_router_backward"}


@pytest.mark.parametrize("call", list(CALLS))
def test_calls_that_are_right_reach_the_library(lib, call):
    call()
    assert lib.calls[-1][0] == CALLS[call]


@pytest.mark.parametrize("call,bad", [
    (norm, dict(res=buf((T, D)))),                              # not h's type
    (norm, dict(h=None)),                                       # a residual without a sum
    (norm, dict(res=None)),                                     # h is x then, of x's type
    (norm, dict(scales=buf((T, 1)))),
    (norm, dict(codes=buf((T, D), torch.int8))),
    (norm, dict(y=buf((T, D)))),
    (norm, dict(x=buf((D, T)).t())),
    (norm, dict(x=buf((T, D), torch.float16))),
    (norm, dict(gamma=buf(D, BF16))),
    (norm_backward, dict(dres=buf((T, D)))),
    (norm_backward, dict(dx=buf((T, D)))),
    (norm_backward, dict(rstd=buf(T - 1))),
    (norm_backward, dict(scratch=buf(SCRATCH - 1, torch.uint8))),
    (weights, dict(W=buf((E, D, N)))),
    (weights, dict(scales=buf((E, 4, 2)))),                     # three blocks in one half
    (weights, dict(halves=2)),                                  # four in two
    (weights, dict(halves=3)),
    (weights, dict(codes=buf((E, N, D), BF16))),
    (product, dict(A=buf((T, D), E4M3))),                       # token rows without perm
    (product, dict(perm=buf(S, I32))),                          # rows in order with it
    (product, dict(perm=buf(S, torch.int64), A=buf((T, D), E4M3), A_scales=buf((T, 2)))),
    (product, dict(A_scales=buf((S, 1)))),
    (product, dict(W_scales=buf((E, 4, 2)))),                   # laid out for two halves
    (product, dict(Y=buf((S, N), BF16))),
    (product, dict(workspace=buf(WORKSPACE - 1, torch.uint8))),
    (product, dict(dev_status=buf(3, I32))),
    (product, dict(offsets=buf(E, I32))),
    (swiglu, dict(W1_scales=buf((E, 3, 2)))),
    (swiglu, dict(H=buf((S, N), E4M3))),
    (swiglu, dict(H=buf((S, N // 2), BF16))),
    (swiglu, dict(H_scales=buf((S, 1)))),
    (losses, dict(load=buf((1, E), I32))),                      # two sequences
    (losses, dict(tokens=buf(2, I32))),
    (losses, dict(seq_len=-1)),
    (losses, dict(seq_len=1 << 32)),
    (losses, dict(mask=buf(T, I32))),
    (losses, dict(topk_idx=buf((T, K), torch.int64))),
    (losses, dict(loss=buf(1))),
    (losses_backward, dict(dlogits=buf((T, E), BF16))),
    (losses_backward, dict(dtopk_w=buf((T, K + 1)))),
    (losses_backward, dict(seq_len=3)),                         # load of one group
])
def test_tensors_that_would_be_misread_are_refused(lib, call, bad):
    with pytest.raises(ValueError):
        call(**bad)
    assert not [c for c in lib.calls if c[0] == CALLS[call]]


@pytest.mark.parametrize("call", [norm, weights, product, losses])
def test_tensors_of_another_device_are_refused(lib, call, monkeypatch):
    global plan
    there = plan
    monkeypatch.setitem(globals(), "plan", lambda: there(device=0))
    with pytest.raises(ValueError, match="cuda:0"):
        call()


def test_scale_blocks_and_groups():
    assert [binding.scale_blocks(n) for n in (16, 128, 144, 1408)] == [1, 1, 2, 11]
    p = plan()
    assert [binding.loss_groups(p, n) for n in (0, 1, 4, 6, 7)] == [1, 6, 2, 1, 1]


class Planned(Exception):
    """A stand-in's constructor has come as far as its plan."""


@pytest.fixture
def like(monkeypatch):
    def no_plan(*a, **kw):
        raise Planned
    monkeypatch.setattr(binding, "moe_plan", no_plan)
    from moe_token_dispatch_route_gb300 import serving
    v = object.__new__(serving.MoeServeLayer)
    v.T, v.d, v.F, v.E, v.k, v.eps, v.route_flags = T, 32, 48, E, K, 1e-6, binding.MOE_ROUTE_SIGMOID
    v.gamma, v.W_r, v.selection_bias, v.device = buf(32), buf((32, E), BF16), None, torch.device("cpu")
    v.weights = (None,) * 4
    return v


def test_what_a_layer_shares_may_be_left_out_or_said_again(like):
    from moe_token_dispatch_route_gb300.serving import MoeServeLayer
    for args, kw in (((None, None, None, None, 0), {}), ((None, None, None, None, None), {}), ((like.gamma, like.W_r, None, None, K), {}),
                     ((None, None, None, None, 0), dict(eps=1e-6, route_flags=binding.MOE_ROUTE_SIGMOID))):
        with pytest.raises(Planned):
            MoeServeLayer(3, *args, like=like, **kw)


@pytest.mark.parametrize("bad", [
    dict(k=K + 1), dict(gamma=buf(32)), dict(W_r=buf((32, E), BF16)), dict(W1=buf((E, 32, 96), BF16)), dict(W2=buf((E, 48, 32), BF16)),
    dict(eps=1e-5), dict(route_flags=binding.MOE_ROUTE_RENORM), dict(route_flags=0), dict(selection_bias=buf(E)),
])
def test_what_a_layer_shares_is_not_dropped_in_silence(like, bad):
    from moe_token_dispatch_route_gb300.serving import MoeServeLayer
    name = next(iter(bad))
    with pytest.raises(ValueError, match=name):
        MoeServeLayer(3, **{**dict(gamma=None, W_r=None, W1=None, W2=None, k=0), **bad}, like=like)
