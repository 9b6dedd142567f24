"""GPU: the data checks look at a call's inputs, also where the call overwrites them."""
import pytest
import torch

import precision_moe_gemm_amd as nv
from precision_moe_gemm_amd import _lib
from tests.gpu_util import step
from tests.test_gpu_checks import checks  # noqa: F401  (the fixture)
from tests.test_gpu_kv_append import call, make as make_append
from tests.test_gpu_norm import make

pytestmark = pytest.mark.gpu
TOP = 3.3895313892515355e38  # the largest bf16


@pytest.mark.parametrize("place", ["x", "residual"])
def test_a_sum_that_overflows_is_no_bad_input(checks, place):
    x, res, w = make(3, 256, 1)
    x[1, 3], res[1, 3] = TOP, TOP
    step(f"checks: the sum in place of {place}")
    r, _, _, _ = nv.mxfp8_add_rmsnorm(x, res, w, sum_out=x if place == "x" else res)
    assert torch.isinf(r[1, 3]) and nv.nvfp4_get_error() == 0


@pytest.mark.parametrize("place", ["x", "residual"])
def test_a_bad_input_of_a_norm_in_place(checks, place):
    x, res, w = make(3, 256, 2)
    (x if place == "x" else res)[2, 100] = float("inf")
    nv.mxfp8_add_rmsnorm(x, res, w, sum_out=x if place == "x" else res)
    assert nv.nvfp4_get_error() == _lib.DATA


def test_a_rotation_that_overflows_is_no_bad_input(checks):
    c = make_append(4, 2, 2, 64, 64, seed=1)
    c["positions"].fill_(1)  # cos + sin of the first pair's angle pass 1
    c["q"][2, 1, 0], c["q"][2, 1, 32] = TOP, TOP
    step("checks: q rotated in place")
    q = call(c, q_out=c["q"])
    assert torch.isinf(q[2, 1]).any() and nv.nvfp4_get_error() == 0


def test_a_bad_query_that_the_rotation_clears(checks):
    """The q row of a token without a position becomes zeros: what stood there was bad all the same."""
    c = make_append(4, 2, 2, 64, 64, seed=2)
    c["slots"][1], c["positions"][1] = -1, -1
    c["q"][1, 0, 7] = float("nan")
    q = call(c, q_out=c["q"])
    assert (q[1] == 0).all() and nv.nvfp4_get_error() == _lib.DATA
