"""The training entry points without a GPU: a missing plan or result pointer is an argument error."""
import ctypes

import pytest

from moe_token_dispatch_route_gb300 import binding

NAMES = ("moe_backward_scratch", "moe_layernorm", "moe_layernorm_backward", "moe_swiglu_checkpoint",
         "moe_swiglu_checkpoint_backward", "moe_combine_backward", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad")


@pytest.fixture(scope="module")
def lib():
    from moe_token_dispatch_route_gb300 import build
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("name", NAMES)
def test_a_missing_plan_is_refused(lib, name):
    fn = getattr(lib, name)
    zero = {ctypes.c_int32: 0, ctypes.c_float: 1e-5}
    assert fn(*[zero.get(t) for t in fn.argtypes]) == binding.MOE_ERR_INVALID_ARG


def test_checkpoint_blocks():
    assert [binding.checkpoint_blocks(F) for F in (8, 120, 128, 136, 1408)] == [1, 1, 1, 2, 11]
