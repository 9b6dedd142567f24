"""GPU: mxfp8_add_rmsnorm where a row's sum is infinite or NaN, against the formula.

1 / sqrt(inf) is 0: the finite elements of such a row become zeros, the infinite ones inf * 0 = NaN.  A NaN
in a row makes its mean and every element NaN."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from precision_moe_gemm_amd import synth
from tests.attn_check import add_rmsnorm
from tests.gpu_util import step, u8
from tests.test_gpu_norm import DEV, make

pytestmark = pytest.mark.gpu
TOP = 3.3895313892515355e38  # the largest bf16


@pytest.mark.parametrize("cols", [32, 256, 1024, 7168])
def test_infinite_and_nan_sums(orc, cols):
    x, res, w = make(7, cols, cols)
    x[1, 5], res[1, 5] = TOP, TOP              # finite parts whose sum passes bf16's range
    x[2, cols - 1], res[2, cols - 1] = -TOP, -TOP
    x[3, 0] = float("inf")
    x[4, 9] = float("nan")
    x[5, 7], res[5, 7] = float("inf"), -float("inf")
    step(f"norm of infinite rows of {cols}")
    r, y, fp8, e8 = nv.mxfp8_add_rmsnorm(x, res, w, 1e-6, want_y=True)
    wr, wy = add_rmsnorm(x, res, w, 1e-6)
    bad = wy.isnan()
    want = [0, 1, 1, 1, cols, cols, 0]
    assert bad.sum(1).tolist() == want and torch.isinf(wr).sum(1).tolist() == [0, 1, 1, 1, 0, 0, 0]  # (the formula's)
    r, y = r.cpu(), y.cpu()
    assert torch.equal(r.isnan(), wr.isnan()) and torch.equal(r[~r.isnan()], wr[~wr.isnan()])
    assert torch.equal(y.isnan(), bad)
    assert torch.equal(y[~bad].view(torch.int16), wy[~bad].view(torch.int16))
    # blocks of 32 without a NaN: the encode's bytes
    clean = ~bad.unflatten(1, (-1, 32)).any(2)
    q, e = orc.mxfp8_encode(np.ascontiguousarray(synth.bits(torch.where(bad, 0, wy))))
    np.testing.assert_array_equal(u8(e8)[clean.numpy()], np.asarray(e)[clean.numpy()])
    np.testing.assert_array_equal(u8(fp8).reshape(7, -1, 32)[clean.numpy()],
                                  np.asarray(q).reshape(7, -1, 32)[clean.numpy()])
