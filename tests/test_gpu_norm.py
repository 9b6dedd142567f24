"""GPU parity: mxfp8_add_rmsnorm against its documented steps and the oracle's MXFP8 encode, byte for byte."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from precision_moe_gemm_amd import synth
from tests.attn_check import add_rmsnorm
from tests.gpu_util import step, u8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(rows, cols, seed=0, spread=0.7):
    g = torch.Generator().manual_seed(seed)
    ch = torch.exp(spread * torch.randn(cols, generator=g))
    x = (torch.randn((rows, cols), generator=g) * ch).bfloat16().to(DEV)
    res = (3 * torch.randn((rows, cols), generator=g) * ch).bfloat16().to(DEV)
    w = (1 + 0.3 * torch.randn(cols, generator=g)).bfloat16().to(DEV)
    return x, res, w


def check(orc, x, res, w, eps, got):
    r, y, fp8, e8 = got
    wr, wy = add_rmsnorm(x, res, w, eps)
    assert torch.equal(r.cpu().view(torch.int16), wr.view(torch.int16))
    if y is not None:
        assert torch.equal(y.cpu().view(torch.int16), wy.view(torch.int16))
    if fp8 is not None:
        q, e = orc.mxfp8_encode(np.ascontiguousarray(synth.bits(wy)))
        np.testing.assert_array_equal(u8(e8), e)
        np.testing.assert_array_equal(u8(fp8), q)


@pytest.mark.parametrize("cols", [32, 64, 96, 512, 544, 1024, 2048, 2080, 5120, 7168, 8192, 8224, 16384, 20000, 40960, 65536])
@pytest.mark.parametrize("rows", [1, 5])
def test_widths(orc, rows, cols):
    x, res, w = make(rows, cols, cols)
    step(f"norm {rows} x {cols}")
    check(orc, x, res, w, 1e-6, nv.mxfp8_add_rmsnorm(x, res, w, 1e-6, want_y=True))


@pytest.mark.parametrize("rows,cols", [(2, 7168), (300, 256), (1023, 1056), (4097, 512), (2500, 5120), (70000, 32)])
def test_batches(orc, rows, cols):
    x, res, w = make(rows, cols, rows)
    step(f"norm {rows} x {cols}")
    check(orc, x, res, w, 1e-5, nv.mxfp8_add_rmsnorm(x, res, w, 1e-5, want_y=True))


def test_optional_parts(orc):
    x, res, w = make(9, 416, 1)
    check(orc, x, None, w, 1e-6, nv.mxfp8_add_rmsnorm(x, None, w, 1e-6, want_y=True))
    check(orc, x, None, None, 1e-6, nv.mxfp8_add_rmsnorm(x, None, None, 1e-6))
    check(orc, x, res, None, 0.0, nv.mxfp8_add_rmsnorm(x, res, None, 0.0, want_y=True, want_fp8=False))
    copy = torch.empty_like(x)
    got = nv.mxfp8_add_rmsnorm(x, None, w, 1e-6, sum_out=copy)
    assert got[0].data_ptr() == copy.data_ptr() and torch.equal(copy, x)


@pytest.mark.parametrize("alias", ["x", "residual"])
@pytest.mark.parametrize("rows", [3, 3000])
def test_sum_in_place(orc, alias, rows):
    x, res, w = make(rows, 2048, 2)
    x0, r0 = x.clone(), res.clone()
    got = nv.mxfp8_add_rmsnorm(x, res, w, 1e-6, want_y=True, sum_out=x if alias == "x" else res)
    check(orc, x0, r0, w, 1e-6, got)


@pytest.mark.parametrize("rows", [6, 2600])
def test_strides(orc, rows):
    x, res, w = make(rows, 1024, 3)
    wide = torch.randn((rows, 2120), device=DEV).bfloat16()
    wide[:, 8:1032], wide[:, 1040:2064] = x, res
    out = torch.full((rows, 1056), 9.0, dtype=torch.bfloat16, device=DEV)
    got = nv.mxfp8_add_rmsnorm(wide[:, 8:1032], wide[:, 1040:2064], w, 1e-6, sum_out=out[:, 16:1040])
    check(orc, x, res, w, 1e-6, got)
    assert (out[:, :16] == 9).all() and (out[:, 1040:] == 9).all()


@pytest.mark.parametrize("cols", [32, 64, 96, 128, 160, 224, 256, 288])
@pytest.mark.parametrize("rows", [1, 7, 33, 20001])
def test_narrow_rows(orc, rows, cols):
    """Several rows to a wave: odd numbers of them, strided, in place, without a residual or a weight."""
    x, res, w = make(rows, cols, cols + rows)
    step(f"narrow {rows} x {cols}")
    check(orc, x, res, w, 1e-6, nv.mxfp8_add_rmsnorm(x, res, w, 1e-6, want_y=True))
    check(orc, x, None, None, 1e-6, nv.mxfp8_add_rmsnorm(x, None, None, 1e-6, want_y=True))
    wide = torch.full((rows, 2 * cols + 24), 9.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + cols], wide[:, 16 + cols:16 + 2 * cols] = x, res
    got = nv.mxfp8_add_rmsnorm(wide[:, 8:8 + cols], wide[:, 16 + cols:16 + 2 * cols], w, 1e-6,
                               sum_out=wide[:, 8:8 + cols])
    check(orc, x, res, w, 1e-6, got)
    assert (wide[:, :8] == 9).all() and (wide[:, 8 + cols:16 + cols] == 9).all() and (wide[:, 16 + 2 * cols:] == 9).all()


def test_extreme_rows(orc):
    """Zero rows (eps keeps them finite), tiny rows, huge rows, one element only."""
    x, res, w = make(6, 256, 4)
    x[0], res[0] = 0, 0
    x[1], res[1] = x[1] * 1e-30, 0
    x[2], res[2] = x[2] * 1e30, 0
    x[3], res[3] = 0, 0
    x[3, 77] = 5.0
    res[4] = -x[4]
    x[5] = 2.0 ** -133
    res[5] = 0
    for eps in (1e-6, 1e-12):
        check(orc, x, res, w, eps, nv.mxfp8_add_rmsnorm(x, res, w, eps, want_y=True))


def test_empty_and_refusals():
    x, res, w = make(4, 64, 5)
    r, y, q, e = nv.mxfp8_add_rmsnorm(x[:0], res[:0], w)
    assert r.shape == (0, 64) and q.shape == (0, 64) and e.shape == (0, 2)
    for a in ((x.float(), res, w), (x, res[:2], w), (x, res, w[:32]), (x.cpu(), None, None), (x, res.half(), w)):
        with pytest.raises(ValueError):
            nv.mxfp8_add_rmsnorm(*a)
    for a in ((x[:, :48], res[:, :48], w[:48], 1e-6), (x, res, w, -1.0), (x, res, w, float("nan"))):
        with pytest.raises(nv.NVFP4Error):
            nv.mxfp8_add_rmsnorm(*a)


def test_graph_replays(orc):
    x, res, w = make(40, 512, 6)
    nv.mxfp8_add_rmsnorm(x, res, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nv.mxfp8_add_rmsnorm(x, res, w)
    for rep in range(3):
        x.copy_(make(40, 512, 7 + rep)[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(orc, x, res, w, 1e-6, (got[0], None, got[2], got[3]))
