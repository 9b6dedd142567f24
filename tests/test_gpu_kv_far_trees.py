"""GPU parity: attention of trees of drafts over a cache whose codes pass 4 GiB."""
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.attn_check import assert_attention
from tests.gpu_util import step
from tests.test_gpu_kv_attention_tree import DEV, call, make, reference, widened

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
def test_offsets_past_32_bits(D):
    """Pages at the far end: whole row tiles, shares of row tiles, tiles."""
    heads, page = 4, 64
    c = make([20, 3, 40], [150, 200, 300], heads, 2, D, page, seed=71)
    want = reference(c)
    small = c["k_cache"].rows // heads // page
    pool = (5 << 30) // (page * heads * D // 2)
    for name in ("k_cache", "v_cache"):
        s, big = c[name], nv.NVFP4Tensor.empty(pool * page * heads, D, 1, DEV)
        big.packed[0, -s.rows:] = s.packed[0]
        big.scales[0, -s.rows:] = s.scales[0]
        big.global_.copy_(s.global_)
        c[name] = big
    c["table"] = torch.where(c["table"] >= 0, c["table"] + (pool - small), -1).int()
    for x, table in ((c, "its own table"), (widened(c), "a wide table")):
        for max_q in (8, 32, 40, 200):
            what = f"trees past 4 GiB, D={D} max_q={max_q}, {table}"
            step(what)
            out, lse = call(x, max_q)
            torch.cuda.synchronize()
            assert nv.nvfp4_get_error() == 0, what
            assert_attention(out, lse, want, what)
