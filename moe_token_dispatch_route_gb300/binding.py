"""Thin ctypes binding of libmoe_gb300.so (the C ABI in include/moe.h).

Argument marshalling only: tensors are handed over as raw device pointers
together with the current CUDA stream; every step of the path runs in the
library's kernels.  Importing this module does not need a GPU; the first
call loads the library and raises if it has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")
_lib = None

STATUS_NAMES = {
    0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
    4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_CAPACITY", 7: "MOE_ERR_DEVICE",
}
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_CAPACITY = 6
MOE_ERR_DEVICE = 7
MOE_ROUTE_RENORM = 1
MOE_ROUTE_SIGMOID = 2
MOE_OUT_F32 = 0
MOE_OUT_BF16 = 1


class MoeError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call} returned {STATUS_NAMES.get(status, status)}")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
        ("k", ctypes.c_int32), ("N", ctypes.c_int32), ("num_ranks", ctypes.c_int32),
        ("rank_capacity_rows", ctypes.c_int32), ("tile_n", ctypes.c_int32),
        ("producer_ctas", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
        ("timeout_ns", ctypes.c_int64), ("debug_skip_publish", ctypes.c_int32),
        ("route_flags", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
    ]


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32),
        ("stages", ctypes.c_int32), ("num_ctas", ctypes.c_int32), ("producer_ctas", ctypes.c_int32),
        ("sm_count", ctypes.c_int32), ("smem_bytes", ctypes.c_int32), ("max_mtiles", ctypes.c_int32),
        ("route_blocks", ctypes.c_int32), ("workspace_bytes", ctypes.c_int64),
        ("half_tiles", ctypes.c_int32), ("background_scatter", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


EXPORTED = ("moe_plan", "moe_plan_destroy", "moe_plan_info", "moe_route", "moe_dispatch_gemm",
            "moe_read_status", "moe_status_string", "moe_route_noalloc", "moe_combine",
            "moe_router_logits", "moe_route_biased", "moe_dispatch_gemm_swiglu",
            "moe_grouped_gemm", "moe_gather_gemm", "moe_set_trace", "moe_dispatch_gemm_combine",
            "moe_backward_scratch", "moe_layernorm", "moe_layernorm_backward", "moe_swiglu_checkpoint",
            "moe_swiglu_checkpoint_backward", "moe_combine_backward", "moe_grouped_gemm_dgrad",
            "moe_grouped_gemm_wgrad", "moe_rmsnorm", "moe_rmsnorm_backward", "moe_quantize_weights",
            "moe_grouped_gemm_fp8", "moe_grouped_gemm_fp8_swiglu", "moe_balance_scratch", "moe_balance_loss",
            "moe_router_backward")


def load_library(path: str = LIB_PATH):
    """Load libmoe_gb300.so and declare its signatures (raises if it is missing)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first (__graft_entry__.build() or "
            "python moe_token_dispatch_route_gb300/build.py); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, I32, VP = ctypes.POINTER, ctypes.c_int32, ctypes.c_void_p
    lib.moe_plan.argtypes = [P(Shape), ctypes.c_int, P(VP), P(ctypes.c_size_t)]
    lib.moe_plan.restype = I32
    lib.moe_plan_destroy.argtypes = [VP]
    lib.moe_plan_destroy.restype = I32
    lib.moe_plan_info.argtypes = [VP, P(PlanInfo)]
    lib.moe_plan_info.restype = I32
    lib.moe_route.argtypes = [VP] * 10
    lib.moe_route.restype = I32
    lib.moe_route_biased.argtypes = [VP] * 11
    lib.moe_route_biased.restype = I32
    lib.moe_dispatch_gemm.argtypes = [VP] * 10
    lib.moe_dispatch_gemm.restype = I32
    lib.moe_dispatch_gemm_combine.argtypes = [VP] * 12
    lib.moe_dispatch_gemm_combine.restype = I32
    lib.moe_dispatch_gemm_swiglu.argtypes = [VP] * 10
    lib.moe_dispatch_gemm_swiglu.restype = I32
    lib.moe_grouped_gemm.argtypes = [VP] * 8
    lib.moe_grouped_gemm.restype = I32
    lib.moe_gather_gemm.argtypes = [VP] * 9
    lib.moe_gather_gemm.restype = I32
    lib.moe_set_trace.argtypes = [VP, VP, ctypes.c_int64]
    lib.moe_set_trace.restype = I32
    lib.moe_read_status.argtypes = [VP, VP, P(I32)]
    lib.moe_read_status.restype = I32
    lib.moe_router_logits.argtypes = [VP] * 6
    lib.moe_router_logits.restype = I32
    lib.moe_combine.argtypes = [VP] * 6
    lib.moe_combine.restype = I32
    lib.moe_route_noalloc.argtypes = [VP] * 9
    lib.moe_route_noalloc.restype = I32
    F32 = ctypes.c_float
    lib.moe_backward_scratch.argtypes = [VP, P(ctypes.c_size_t)]
    lib.moe_layernorm.argtypes = [VP, VP, I32, VP, VP, F32, VP, VP, VP, VP]
    lib.moe_layernorm_backward.argtypes = [VP, VP, I32, VP, I32] + [VP] * 9
    lib.moe_swiglu_checkpoint.argtypes = [VP] * 6
    lib.moe_swiglu_checkpoint_backward.argtypes = [VP, VP, I32] + [VP] * 5
    lib.moe_combine_backward.argtypes = [VP, VP, I32] + [VP] * 6
    lib.moe_grouped_gemm_dgrad.argtypes = [VP] * 5 + [I32] + [VP] * 3
    lib.moe_grouped_gemm_wgrad.argtypes = [VP] * 5 + [I32, I32] + [VP] * 3
    lib.moe_rmsnorm.argtypes = [VP, VP, I32, VP, I32, VP, F32] + [VP] * 6
    lib.moe_rmsnorm_backward.argtypes = [VP, VP, I32, VP, I32] + [VP] * 7
    lib.moe_quantize_weights.argtypes = [VP, VP, I32, VP, VP, VP]
    lib.moe_grouped_gemm_fp8.argtypes = [VP] * 11
    lib.moe_grouped_gemm_fp8_swiglu.argtypes = [VP] * 12
    lib.moe_balance_scratch.argtypes = [VP, I32, P(ctypes.c_size_t)]
    lib.moe_balance_loss.argtypes = [VP] * 4 + [I32, F32, F32] + [VP] * 5
    lib.moe_router_backward.argtypes = [VP] * 5 + [I32, F32, F32] + [VP] * 4
    for name in EXPORTED[-16:]:  # the training operators, the 8-bit forward pass and the router's losses
        getattr(lib, name).restype = I32
    lib.moe_status_string.argtypes = [I32]
    lib.moe_status_string.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


# the current stream's handle without building a Stream object (1 us of a launch-bound call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, device=None) -> int:
    if stream is None:
        if _raw_stream is not None and device is not None:
            return _raw_stream(device)
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, call: str):
    if rc != MOE_OK:
        raise MoeError(rc, call)


class Plan:
    """Owns a moe_plan_t; `workspace_bytes` and `info` come from the library."""

    def __init__(self, handle: int, workspace_bytes: int, shape: Shape, device: int):
        self.handle = handle
        self.workspace_bytes = workspace_bytes
        self.shape = shape
        self.device = device
        self.T, self.d, self.E, self.N, self.S = shape.T, shape.d, shape.E, shape.N, shape.T * shape.k
        info = PlanInfo()
        _check(load_library().moe_plan_info(handle, ctypes.byref(info)), "moe_plan_info")
        self.info = info.as_dict()
        scratch = ctypes.c_size_t()
        _check(load_library().moe_backward_scratch(handle, ctypes.byref(scratch)), "moe_backward_scratch")
        self.scratch_bytes = scratch.value

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.moe_plan_destroy(h)


def moe_plan(T: int, d: int, E: int, k: int, N: int, num_ranks: int = 1,
             rank_capacity_rows: int = 0, tile_n: int = 0, producer_ctas: int = 0,
             num_ctas: int = 0, timeout_ns: int = 0, debug_skip_publish: int = 0,
             route_flags: int = 0, tile_m: int = 0, out_dtype: int = MOE_OUT_F32,
             device: int | None = None) -> Plan:
    lib = load_library()
    dev = torch.cuda.current_device() if device is None else int(device)
    shape = Shape(T, d, E, k, N, num_ranks, rank_capacity_rows, tile_n, producer_ctas, num_ctas,
                  timeout_ns, debug_skip_publish, route_flags, tile_m, out_dtype)
    handle = ctypes.c_void_p()
    ws = ctypes.c_size_t()
    _check(lib.moe_plan(ctypes.byref(shape), dev, ctypes.byref(handle), ctypes.byref(ws)), "moe_plan")
    return Plan(handle.value, ws.value, shape, dev)


def moe_route(plan: Plan, logits, topk_idx, topk_w, counts, offsets, perm, dest, workspace,
              stream=None) -> None:
    rc = load_library().moe_route(plan.handle, _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
                                  _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(dest),
                                  _ptr(workspace), _stream(stream, plan.device))
    _check(rc, "moe_route")


def moe_route_biased(plan: Plan, logits, selection_bias, topk_idx, topk_w, counts, offsets, perm,
                     dest, workspace, stream=None) -> None:
    """moe_route ranking experts by logit + selection_bias[e]; gates from the logits."""
    rc = load_library().moe_route_biased(plan.handle, _ptr(logits), _ptr(selection_bias),
                                         _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
                                         _ptr(offsets), _ptr(perm), _ptr(dest), _ptr(workspace),
                                         _stream(stream, plan.device))
    _check(rc, "moe_route_biased")


def moe_route_noalloc(plan: Plan, logits, topk_idx, topk_w, counts, offsets, perm, dest,
                      stream=None) -> None:
    """moe_route without a workspace: the library's static device scratch is used
    instead (for callers that cannot allocate device memory)."""
    rc = load_library().moe_route_noalloc(plan.handle, _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
                                          _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(dest),
                                          _stream(stream, plan.device))
    _check(rc, "moe_route_noalloc")


def moe_dispatch_gemm(plan: Plan, x, offsets, perm, W, recv: Sequence, Y, workspace, dev_status,
                      stream=None) -> None:
    arr = (ctypes.c_void_p * max(1, len(recv)))(*[_ptr(r) for r in recv])
    rc = load_library().moe_dispatch_gemm(plan.handle, _ptr(x), _ptr(offsets), _ptr(perm), _ptr(W),
                                          ctypes.cast(arr, ctypes.c_void_p), _ptr(Y),
                                          _ptr(workspace), _ptr(dev_status),
                                          _stream(stream, plan.device))
    _check(rc, "moe_dispatch_gemm")


def moe_dispatch_gemm_combine(plan: Plan, x, offsets, perm, dest, topk_w, W, recv: Sequence, out, workspace,
                              dev_status, stream=None) -> None:
    """Fused dispatch + grouped GEMM + combine: out[t] = sum_j w[t,j] * (x[t] W[e_j]), summed in
    ascending expert order (no Y)."""
    arr = (ctypes.c_void_p * max(1, len(recv)))(*[_ptr(r) for r in recv])
    rc = load_library().moe_dispatch_gemm_combine(plan.handle, _ptr(x), _ptr(offsets), _ptr(perm), _ptr(dest),
                                                  _ptr(topk_w), _ptr(W), ctypes.cast(arr, ctypes.c_void_p),
                                                  _ptr(out), _ptr(workspace), _ptr(dev_status),
                                                  _stream(stream, plan.device))
    _check(rc, "moe_dispatch_gemm_combine")


def dispatch_gemm_combine(plan: Plan, x, W, bufs: "MoeBuffers", out, stream=None):
    moe_dispatch_gemm_combine(plan, x, bufs.offsets, bufs.perm, bufs.dest, bufs.topk_w, W, bufs.recv, out,
                              bufs.workspace, bufs.status, stream)


def moe_dispatch_gemm_swiglu(plan: Plan, x, offsets, perm, W1, recv: Sequence, H, workspace,
                             dev_status, stream=None) -> None:
    """Fused dispatch + gated up-projection: H = silu(x W1_gate) * (x W1_up), bf16."""
    arr = (ctypes.c_void_p * max(1, len(recv)))(*[_ptr(r) for r in recv])
    rc = load_library().moe_dispatch_gemm_swiglu(plan.handle, _ptr(x), _ptr(offsets), _ptr(perm),
                                                 _ptr(W1), ctypes.cast(arr, ctypes.c_void_p),
                                                 _ptr(H), _ptr(workspace), _ptr(dev_status),
                                                 _stream(stream, plan.device))
    _check(rc, "moe_dispatch_gemm_swiglu")


def moe_grouped_gemm(plan: Plan, A, offsets, W, Y, workspace, dev_status, stream=None) -> None:
    """Per-expert grouped GEMM on rows already in destination order (no scatter)."""
    rc = load_library().moe_grouped_gemm(plan.handle, _ptr(A), _ptr(offsets), _ptr(W), _ptr(Y),
                                         _ptr(workspace), _ptr(dev_status),
                                         _stream(stream, plan.device))
    _check(rc, "moe_grouped_gemm")


def moe_gather_gemm(plan: Plan, x, offsets, perm, W, Y, workspace, dev_status, stream=None) -> None:
    """Grouped GEMM whose A rows are gathered from x by perm (no receive buffers)."""
    rc = load_library().moe_gather_gemm(plan.handle, _ptr(x), _ptr(offsets), _ptr(perm), _ptr(W),
                                        _ptr(Y), _ptr(workspace), _ptr(dev_status),
                                        _stream(stream, plan.device))
    _check(rc, "moe_gather_gemm")


def gather_gemm(plan: Plan, x, W, bufs: "MoeBuffers", stream=None):
    moe_gather_gemm(plan, x, bufs.offsets, bufs.perm, W, bufs.Y, bufs.workspace, bufs.status, stream)


TRACE_WORDS = 8
TRACE_FIELDS = ("start", "scatter_end", "first_tile", "flag_wait_ns", "tiles", "issue_end", "end", "role")


def moe_set_trace(plan: Plan, trace) -> None:
    """Per-CTA timing records of later GEMM launches into `trace` (a device int64
    tensor of at least sm_count * 8 words), or None to stop."""
    nbytes = 0 if trace is None else trace.numel() * trace.element_size()
    _check(load_library().moe_set_trace(plan.handle, _ptr(trace), nbytes), "moe_set_trace")


def moe_router_logits(plan: Plan, x, W_r, bias, logits, stream=None) -> None:
    rc = load_library().moe_router_logits(plan.handle, _ptr(x), _ptr(W_r), _ptr(bias), _ptr(logits),
                                          _stream(stream, plan.device))
    _check(rc, "moe_router_logits")


def moe_combine(plan: Plan, Y, topk_w, dest, out, stream=None) -> None:
    rc = load_library().moe_combine(plan.handle, _ptr(Y), _ptr(topk_w), _ptr(dest), _ptr(out),
                                    _stream(stream, plan.device))
    _check(rc, "moe_combine")


# ---------------------------------------------------------------- training operators

_DTYPES = {torch.float32: MOE_OUT_F32, torch.bfloat16: MOE_OUT_BF16}


_F32, _BF16 = torch.float32, torch.bfloat16
_IS_F32, _IS_BF16, _IS_EITHER, _IS_I32, _IS_I8 = (_F32,), (_BF16,), (_BF16, _F32), (torch.int32,), (torch.int8,)


def _arg(call: str, plan: Plan, name: str, t, numel: int, dtypes: tuple) -> int:
    """Device pointer of a dense tensor on the plan's device with `numel` elements and one of
    `dtypes`; the C ABI sees addresses alone, so a tensor it would misread is refused here."""
    if t is None:
        raise ValueError(f"{call}: {name} is missing")
    if t.dtype in dtypes and t.numel() == numel and t.get_device() == plan.device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise ValueError(f"{call}: {name} is {t.dtype}, wanted {' or '.join(str(d) for d in dtypes)}")
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{call}: {name} must be dense with {numel} elements, got {tuple(t.shape)}"
                         f"{'' if t.is_contiguous() else ', strided'}")
    raise ValueError(f"{call}: {name} is on {t.device}, the plan on cuda:{plan.device}")


def _opt(call: str, plan: Plan, name: str, t, numel: int, dtypes: tuple) -> int | None:
    if t is None:
        return None
    if t.dtype in dtypes and t.numel() == numel and t.get_device() == plan.device and t.is_contiguous():
        return t.data_ptr()
    return _arg(call, plan, name, t, numel, dtypes)


def _buf(call: str, plan: Plan, name: str, t, nbytes: int) -> int | None:
    """Device pointer of a buffer that the kernels write without looking at its size: dense, on the plan's device, at
    least `nbytes` long (one that was made for a smaller plan would be written past its end).  An int is an
    address that the caller answers for; a missing buffer is the library's to refuse."""
    if t is None or isinstance(t, int):
        return t
    if t.nbytes >= nbytes and t.get_device() == plan.device and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != plan.device:
        raise ValueError(f"{call}: {name} is on {t.device}, the plan on cuda:{plan.device}")
    raise ValueError(f"{call}: {name} must be dense with at least {nbytes} bytes, has {t.nbytes}"
                     f"{'' if t.is_contiguous() else ', strided'}")


def backward_scratch(plan: Plan, device=None) -> torch.Tensor:
    """Zeroed scratch of moe_layernorm_backward (the caller keeps it, like the workspace)."""
    return torch.zeros(plan.scratch_bytes, dtype=torch.uint8,
                       device=torch.device("cuda", plan.device) if device is None else device)


def moe_layernorm(plan: Plan, x, gamma, beta, eps: float, y, mean=None, rstd=None, stream=None) -> None:
    """y = (x - mean) rstd gamma + beta over the plan's T rows of width d; gamma, beta, mean and
    rstd may be None."""
    c = "moe_layernorm"
    d, T = plan.d, plan.T
    n = T * d
    _check(load_library().moe_layernorm(
        plan.handle, _arg(c, plan, "x", x, n, _IS_EITHER), _DTYPES[x.dtype],
        _opt(c, plan, "gamma", gamma, d, _IS_F32), _opt(c, plan, "beta", beta, d, _IS_F32),
        eps, _arg(c, plan, "y", y, n, _IS_BF16), _opt(c, plan, "mean", mean, T, _IS_F32),
        _opt(c, plan, "rstd", rstd, T, _IS_F32), _stream(stream, plan.device)), c)


def moe_layernorm_backward(plan: Plan, dy, x, gamma, mean, rstd, dres, dx, dgamma, dbeta, scratch,
                           stream=None) -> None:
    """Gradient of moe_layernorm; dres (added to dx), gamma, dgamma and dbeta may be None."""
    c = "moe_layernorm_backward"
    d, T = plan.d, plan.T
    n = T * d
    px = _arg(c, plan, "x", x, n, _IS_EITHER)
    _check(load_library().moe_layernorm_backward(
        plan.handle, _arg(c, plan, "dy", dy, n, _IS_EITHER), _DTYPES[dy.dtype], px, _DTYPES[x.dtype],
        _opt(c, plan, "gamma", gamma, d, _IS_F32), _arg(c, plan, "mean", mean, T, _IS_F32),
        _arg(c, plan, "rstd", rstd, T, _IS_F32), _opt(c, plan, "dres", dres, n, (x.dtype,)),
        _arg(c, plan, "dx", dx, n, (x.dtype,)), _opt(c, plan, "dgamma", dgamma, d, _IS_F32),
        _opt(c, plan, "dbeta", dbeta, d, _IS_F32),
        None if dgamma is None and dbeta is None else _buf(c, plan, "scratch", scratch, plan.scratch_bytes),
        _stream(stream, plan.device)), c)


def _out_dtype(plan: Plan):
    return _IS_BF16 if plan.shape.out_dtype == MOE_OUT_BF16 else _IS_F32


def checkpoint_blocks(F: int) -> int:
    """Scales of one half row of the 8-bit checkpoint: blocks of 128 columns."""
    return (F + 127) // 128


def moe_swiglu_checkpoint(plan: Plan, GU, H, codes, scales, stream=None) -> None:
    """H = silu(gate) * up (H may be None), and GU in 8 bits: int8 codes [S][2F] and fp32 scales
    [S][2 * checkpoint_blocks(F)]."""
    c = "moe_swiglu_checkpoint"
    S, F = plan.S, plan.N // 2
    _check(load_library().moe_swiglu_checkpoint(
        plan.handle, _arg(c, plan, "GU", GU, S * 2 * F, _out_dtype(plan)),
        _opt(c, plan, "H", H, S * F, _IS_BF16), _arg(c, plan, "codes", codes, S * 2 * F, _IS_I8),
        _arg(c, plan, "scales", scales, S * 2 * checkpoint_blocks(F), _IS_F32), _stream(stream, plan.device)), c)


def moe_swiglu_checkpoint_backward(plan: Plan, dH, codes, scales, H, dGU, stream=None) -> None:
    """dGU from dH and the 8-bit checkpoint, and the activation H again (H may be None)."""
    c = "moe_swiglu_checkpoint_backward"
    S, F = plan.S, plan.N // 2
    _check(load_library().moe_swiglu_checkpoint_backward(
        plan.handle, _arg(c, plan, "dH", dH, S * F, _IS_EITHER), _DTYPES[dH.dtype],
        _arg(c, plan, "codes", codes, S * 2 * F, _IS_I8),
        _arg(c, plan, "scales", scales, S * 2 * checkpoint_blocks(F), _IS_F32),
        _opt(c, plan, "H", H, S * F, _IS_BF16), _arg(c, plan, "dGU", dGU, S * 2 * F, _IS_BF16),
        _stream(stream, plan.device)), c)


def moe_combine_backward(plan: Plan, dout, Y, topk_w, dest, dY, dtopk_w, stream=None) -> None:
    """dY[dest[t,j]] = topk_w[t,j] dout[t] and dtopk_w[t,j] = <dout[t], Y[dest[t,j]]>."""
    c = "moe_combine_backward"
    S, N = plan.S, plan.N
    _check(load_library().moe_combine_backward(
        plan.handle, _arg(c, plan, "dout", dout, plan.T * N, _IS_EITHER), _DTYPES[dout.dtype],
        _arg(c, plan, "Y", Y, S * N, _out_dtype(plan)), _arg(c, plan, "topk_w", topk_w, S, _IS_F32),
        _arg(c, plan, "dest", dest, S, _IS_I32), _arg(c, plan, "dY", dY, S * N, _IS_BF16),
        _arg(c, plan, "dtopk_w", dtopk_w, S, _IS_F32), _stream(stream, plan.device)), c)


def moe_grouped_gemm_dgrad(plan: Plan, dY, offsets, W, dA, workspace, dev_status, stream=None) -> None:
    """dA[i] = dY[i] W[e(i)]^T, fp32 or bf16 by dA's type."""
    c = "moe_grouped_gemm_dgrad"
    S, N = plan.S, plan.N
    _check(load_library().moe_grouped_gemm_dgrad(
        plan.handle, _arg(c, plan, "dY", dY, S * N, _IS_BF16), _arg(c, plan, "offsets", offsets, plan.E + 1, _IS_I32),
        _arg(c, plan, "W", W, plan.E * plan.d * N, _IS_BF16), _arg(c, plan, "dA", dA, S * plan.d, _IS_EITHER),
        _DTYPES[dA.dtype], _buf(c, plan, "workspace", workspace, plan.workspace_bytes),
        _buf(c, plan, "dev_status", dev_status, 16), _stream(stream, plan.device)), c)


def moe_grouped_gemm_wgrad(plan: Plan, A, dY, offsets, dW, workspace, dev_status, accumulate: bool = False,
                           stream=None) -> None:
    """dW[e] = A_e^T dY_e (accumulate: added to dW, fp32), fp32 or bf16 by dW's type."""
    c = "moe_grouped_gemm_wgrad"
    S, N = plan.S, plan.N
    _check(load_library().moe_grouped_gemm_wgrad(
        plan.handle, _arg(c, plan, "A", A, S * plan.d, _IS_BF16), _arg(c, plan, "dY", dY, S * N, _IS_BF16),
        _arg(c, plan, "offsets", offsets, plan.E + 1, _IS_I32),
        _arg(c, plan, "dW", dW, plan.E * plan.d * N, _IS_EITHER), _DTYPES[dW.dtype], int(accumulate),
        _buf(c, plan, "workspace", workspace, plan.workspace_bytes), _buf(c, plan, "dev_status", dev_status, 16),
        _stream(stream, plan.device)), c)


# ---------------------------------------------------------------- 8-bit forward pass

_IS_E4M3 = (torch.float8_e4m3fn, torch.uint8)


def scale_blocks(n: int) -> int:
    """Scales of n columns stored in 8 bits: blocks of 128."""
    return (n + 127) // 128


def moe_rmsnorm(plan: Plan, x, res, gamma, eps: float, h, y, codes=None, scales=None, rstd=None, stream=None) -> None:
    """h = x + res, y = h rstd gamma over the plan's T rows of width d; y in bf16 and (or) in 8 bits as e4m3 codes
    [T][d] and fp32 scales [T][scale_blocks(d)].  res, gamma, y or codes and scales, and rstd may be None; h may be res, and
    None without one."""
    c = "moe_rmsnorm"
    d, T = plan.d, plan.T
    n = T * d
    px = _arg(c, plan, "x", x, n, _IS_EITHER)
    kind = (x.dtype,) if res is None else _IS_EITHER
    ph = _opt(c, plan, "h", h, n, kind) if res is None else _arg(c, plan, "h", h, n, kind)
    hd = x.dtype if h is None else h.dtype
    _check(load_library().moe_rmsnorm(
        plan.handle, px, _DTYPES[x.dtype], _opt(c, plan, "res", res, n, (hd,)), _DTYPES[hd],
        _opt(c, plan, "gamma", gamma, d, _IS_F32), eps, ph, _opt(c, plan, "y", y, n, _IS_BF16),
        _opt(c, plan, "codes", codes, n, _IS_E4M3), _opt(c, plan, "scales", scales, T * scale_blocks(d), _IS_F32),
        _opt(c, plan, "rstd", rstd, T, _IS_F32), _stream(stream, plan.device)), c)


def moe_rmsnorm_backward(plan: Plan, dy, h, gamma, rstd, dres, dx, dgamma, scratch, stream=None) -> None:
    """Gradient of moe_rmsnorm with respect to h; dres (added to dx), gamma and dgamma may be None."""
    c = "moe_rmsnorm_backward"
    d, T = plan.d, plan.T
    n = T * d
    ph = _arg(c, plan, "h", h, n, _IS_EITHER)
    _check(load_library().moe_rmsnorm_backward(
        plan.handle, _arg(c, plan, "dy", dy, n, _IS_EITHER), _DTYPES[dy.dtype], ph, _DTYPES[h.dtype],
        _opt(c, plan, "gamma", gamma, d, _IS_F32), _arg(c, plan, "rstd", rstd, T, _IS_F32),
        _opt(c, plan, "dres", dres, n, (h.dtype,)), _arg(c, plan, "dx", dx, n, (h.dtype,)),
        _opt(c, plan, "dgamma", dgamma, d, _IS_F32),
        None if dgamma is None else _buf(c, plan, "scratch", scratch, plan.scratch_bytes), _stream(stream, plan.device)), c)


def _weight_scales(plan: Plan, halves: int) -> int:
    return plan.E * halves * scale_blocks(plan.N // halves) * scale_blocks(plan.d)


def moe_quantize_weights(plan: Plan, W, codes, scales, halves: int = 1, stream=None) -> None:
    """W bf16 [E][d][N] as e4m3 codes [E][N][d] and fp32 scales [E][halves * scale_blocks(N / halves)][scale_blocks(d)];
    halves is 2 for the gate and up projections of a gated layer."""
    c = "moe_quantize_weights"
    n = plan.E * plan.d * plan.N
    if halves not in (1, 2):
        raise ValueError(f"{c}: halves is 1 or 2, got {halves}")
    _check(load_library().moe_quantize_weights(
        plan.handle, _arg(c, plan, "W", W, n, _IS_BF16), halves, _arg(c, plan, "codes", codes, n, _IS_E4M3),
        _arg(c, plan, "scales", scales, _weight_scales(plan, halves), _IS_F32), _stream(stream, plan.device)), c)


def _fp8_operands(c: str, plan: Plan, A, A_scales, perm, offsets, W, W_scales, halves: int) -> list:
    rows = plan.S if perm is None else plan.T
    return [_arg(c, plan, "A", A, rows * plan.d, _IS_E4M3),
            _arg(c, plan, "A_scales", A_scales, rows * scale_blocks(plan.d), _IS_F32),
            _opt(c, plan, "perm", perm, plan.S, _IS_I32), _arg(c, plan, "offsets", offsets, plan.E + 1, _IS_I32),
            _arg(c, plan, "W", W, plan.E * plan.d * plan.N, _IS_E4M3),
            _arg(c, plan, "W_scales", W_scales, _weight_scales(plan, halves), _IS_F32)]


def moe_grouped_gemm_fp8(plan: Plan, A, A_scales, perm, offsets, W, W_scales, Y, workspace, dev_status, stream=None) -> None:
    """Per-expert product on 8-bit rows and weights: Y[i] = A[r] W[e(i)]^T, r = i or (with perm) the row's token."""
    c = "moe_grouped_gemm_fp8"
    _check(load_library().moe_grouped_gemm_fp8(
        plan.handle, *_fp8_operands(c, plan, A, A_scales, perm, offsets, W, W_scales, 1),
        _arg(c, plan, "Y", Y, plan.S * plan.N, _out_dtype(plan)),
        _buf(c, plan, "workspace", workspace, plan.workspace_bytes), _buf(c, plan, "dev_status", dev_status, 16),
        _stream(stream, plan.device)), c)


def moe_grouped_gemm_fp8_swiglu(plan: Plan, A, A_scales, perm, offsets, W1, W1_scales, H, H_scales, workspace, dev_status,
                                stream=None) -> None:
    """moe_grouped_gemm_fp8 for gate and up projections: H = silu(gate) * up as e4m3 codes [S][F] and fp32 scales
    [S][scale_blocks(F)]."""
    c = "moe_grouped_gemm_fp8_swiglu"
    F = plan.N // 2
    _check(load_library().moe_grouped_gemm_fp8_swiglu(
        plan.handle, *_fp8_operands(c, plan, A, A_scales, perm, offsets, W1, W1_scales, 2),
        _arg(c, plan, "H", H, plan.S * F, _IS_E4M3), _arg(c, plan, "H_scales", H_scales, plan.S * scale_blocks(F), _IS_F32),
        _buf(c, plan, "workspace", workspace, plan.workspace_bytes), _buf(c, plan, "dev_status", dev_status, 16),
        _stream(stream, plan.device)), c)


# ---------------------------------------------------------------- router's losses

_IS_MASK = (torch.bool, torch.uint8)


def loss_groups(plan: Plan, seq_len: int) -> int:
    """Groups of tokens that the balance loss is taken over: sequences of seq_len, or (0) all tokens."""
    if not 0 <= seq_len < 1 << 31:
        raise ValueError(f"seq_len must be 0 or a number of tokens, got {seq_len}")
    return max(1, -(-plan.T // seq_len)) if seq_len else 1


def _balance_scratch_bytes(plan: Plan, seq_len: int) -> int:
    known = plan.__dict__.setdefault("balance_scratch_bytes", {})  # of the plan's shape and seq_len alone
    if seq_len in known:
        return known[seq_len]
    n = ctypes.c_size_t()
    _check(load_library().moe_balance_scratch(plan.handle, seq_len, ctypes.byref(n)), "moe_balance_scratch")
    known[seq_len] = n.value
    return n.value


def balance_scratch(plan: Plan, seq_len: int = 0, device=None) -> torch.Tensor:
    """Scratch of moe_balance_loss (the caller keeps it, like the workspace)."""
    return torch.zeros(_balance_scratch_bytes(plan, seq_len), dtype=torch.uint8,
                       device=torch.device("cuda", plan.device) if device is None else device)


def moe_balance_loss(plan: Plan, logits, topk_idx, mask, seq_len: int, balance: float, z: float, loss, load, tokens, scratch,
                     stream=None) -> None:
    """loss[0], loss[1]: the router's balance loss over sequences of seq_len tokens (0: all in one) and its z loss, times
    their coefficients; load int32 [groups][E]: counted picks; tokens int32 [groups + 1]: counted tokens, at last all.
    mask (bool or uint8 [T], 0: the token does not count) may be None."""
    c = "moe_balance_loss"
    G = loss_groups(plan, seq_len)
    _check(load_library().moe_balance_loss(
        plan.handle, _arg(c, plan, "logits", logits, plan.T * plan.E, _IS_F32),
        _arg(c, plan, "topk_idx", topk_idx, plan.S, _IS_I32), _opt(c, plan, "mask", mask, plan.T, _IS_MASK), seq_len,
        balance, z, _arg(c, plan, "loss", loss, 2, _IS_F32), _arg(c, plan, "load", load, G * plan.E, _IS_I32),
        _arg(c, plan, "tokens", tokens, G + 1, _IS_I32),
        _buf(c, plan, "scratch", scratch, _balance_scratch_bytes(plan, seq_len)), _stream(stream, plan.device)), c)


def moe_router_backward(plan: Plan, logits, topk_idx, dtopk_w, mask, seq_len: int, balance: float, z: float, load, tokens,
                        dlogits, stream=None) -> None:
    """dlogits of the losses (load and tokens from moe_balance_loss; None where their coefficients are 0) and, with
    dtopk_w, of the gates."""
    c = "moe_router_backward"
    G = loss_groups(plan, seq_len)
    n = plan.T * plan.E
    _check(load_library().moe_router_backward(
        plan.handle, _arg(c, plan, "logits", logits, n, _IS_F32), _opt(c, plan, "topk_idx", topk_idx, plan.S, _IS_I32),
        _opt(c, plan, "dtopk_w", dtopk_w, plan.S, _IS_F32), _opt(c, plan, "mask", mask, plan.T, _IS_MASK), seq_len,
        balance, z, _opt(c, plan, "load", load, G * plan.E, _IS_I32), _opt(c, plan, "tokens", tokens, G + 1, _IS_I32),
        _arg(c, plan, "dlogits", dlogits, n, _IS_F32), _stream(stream, plan.device)), c)


def moe_read_status(dev_status, stream=None) -> tuple[int, list[int]]:
    out = (ctypes.c_int32 * 4)()
    rc = load_library().moe_read_status(_ptr(dev_status), _stream(stream), out)
    return rc, list(out)


class MoeBuffers:
    """Device buffers of one layer shape, allocated with PyTorch (the caller's
    side of the ABI): routing outputs, R receive buffers, the GEMM output, workspace,
    status.  out="Y": fp32 Y [S][N] (moe_dispatch_gemm); out="H": bf16 H [S][N/2]
    (moe_dispatch_gemm_swiglu)."""

    def __init__(self, plan: Plan, device="cuda", out: str = "Y"):
        s = plan.shape
        S = s.T * s.k
        R = s.num_ranks or 1
        cap = s.rank_capacity_rows or S
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.topk_idx = torch.empty(s.T, s.k, **i32)
        self.topk_w = torch.empty(s.T, s.k, dtype=torch.float32, device=dev)
        self.counts = torch.empty(s.E, **i32)
        self.offsets = torch.empty(s.E + 1, **i32)
        self.perm = torch.empty(S, **i32)
        self.dest = torch.empty(S, **i32)
        self.recv = [torch.empty(max(cap, 1), s.d, dtype=torch.bfloat16, device=dev) for _ in range(R)]
        y_dtype = torch.bfloat16 if s.out_dtype == MOE_OUT_BF16 else torch.float32
        self.Y = torch.empty(S, s.N, dtype=y_dtype, device=dev) if out == "Y" else None
        self.H = torch.empty(S, s.N // 2, dtype=torch.bfloat16, device=dev) if out == "H" else None
        self.workspace = torch.zeros(plan.workspace_bytes // 4 + 64, dtype=torch.int32, device=dev)
        self.status = torch.zeros(4, **i32)


def route(plan: Plan, logits, bufs: MoeBuffers, stream=None, selection_bias=None):
    moe_route_biased(plan, logits, selection_bias, bufs.topk_idx, bufs.topk_w, bufs.counts,
                     bufs.offsets, bufs.perm, bufs.dest, bufs.workspace, stream)


def dispatch_gemm(plan: Plan, x, W, bufs: MoeBuffers, stream=None):
    moe_dispatch_gemm(plan, x, bufs.offsets, bufs.perm, W, bufs.recv, bufs.Y, bufs.workspace,
                      bufs.status, stream)


def dispatch_gemm_swiglu(plan: Plan, x, W1, bufs: MoeBuffers, stream=None):
    moe_dispatch_gemm_swiglu(plan, x, bufs.offsets, bufs.perm, W1, bufs.recv, bufs.H,
                             bufs.workspace, bufs.status, stream)


def forward(plan: Plan, logits, x, W, bufs: MoeBuffers, stream=None):
    """One pass of the whole path: routing, then the fused dispatch + grouped GEMM."""
    route(plan, logits, bufs, stream)
    dispatch_gemm(plan, x, W, bufs, stream)
