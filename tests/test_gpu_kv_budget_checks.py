"""The data checks with the operators for trees and bounded caches: queries and globals are looked at, pages that no
sequence holds may hold anything, and results do not change."""
import pytest
import torch

import precision_moe_gemm_amd as nv
from precision_moe_gemm_amd import _lib
from tests import test_gpu_kv_attention_tree as tree
from tests import test_gpu_kv_weights as weights
from tests.gpu_util import step

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture
def checks():
    prev = nv.nvfp4_set_checks(True)
    assert nv.nvfp4_get_error() == 0
    yield
    nv.nvfp4_set_checks(prev)
    nv.nvfp4_get_error()


def tree_case():
    return tree.make([5, 20], [90, 64], 2, 4, 128, 16, seed=3), lambda c: tree.call(c)[0]


def weights_case():
    return weights.with_lse(weights.make([5, 20], [90, 64], 2, 4, 128, 16, seed=3)), weights.call


@pytest.mark.parametrize("case", [tree_case, weights_case])
def test_data_checks(checks, case):
    nv.nvfp4_set_checks(False)
    c, call = case()
    want = call(c)
    nv.nvfp4_set_checks(True)
    step(f"checks on: {case.__name__}")
    assert torch.equal(call(c), want)
    assert nv.nvfp4_get_error() == 0
    parts = ["k_cache", "v_cache"] if case is tree_case else ["k_cache"]
    for name in parts:
        old = c[name].global_.clone()
        for bad in (-1.0, float("nan")):
            c[name].global_.fill_(bad)
            step(f"checks on: {case.__name__}, {name}'s global {bad}")
            call(c)
            assert nv.nvfp4_get_error() == _lib.DATA, (name, bad)
        c[name].global_.copy_(old)
    c["q"][7, 2, 3] = float("inf")
    step(f"checks on: {case.__name__}, an infinite query")
    call(c)
    assert nv.nvfp4_get_error() == _lib.DATA


def test_weights_without_query_rows(checks):
    c = weights.make([0, 0], [90, 33], 2, 2, 64, 16, seed=35)
    c["lse"] = torch.empty((0, 4), device=DEV)
    step("checks on: no query rows")
    weights.call(c, max_q=1)
    assert nv.nvfp4_get_error() == 0
