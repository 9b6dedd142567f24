"""GPU: the operators for trees and bounded caches write no byte behind the workspace that the library asks for, and
read none that they have not written."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.cache_check import chosen
from tests.gpu_util import step
from tests.test_gpu_kv_attention_tree import DEV, call, make, widened
from tests.test_gpu_kv_evict import make as select_case

pytestmark = pytest.mark.gpu
GUARD = 1 << 16


def room(need):
    """`need` bytes of 0xFF (NaN) and guard bytes behind."""
    space = torch.full((need + GUARD,), 0xFF, dtype=torch.uint8, device=DEV)
    space[need:] = 0x5A
    return space


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 8), (4, 8), (3, 5), (40, 2)])
@pytest.mark.parametrize("max_q", [1, 8, 16, 64, 200])
def test_trees(D, heads, group, max_q):
    """Row tiles of 16 and 32 rows and tiles of 128 and 256, shares of all of them."""
    c = widened(make([60, 3, 64, 33], [1700, 50, 64, 900], heads, group, D, 16, seed=D + heads))
    n, qh, _ = c["q"].shape
    need = nv.nvfp4_workspace_size(nv._lib.OP_KV_ATTENTION_TREE, n, qh, heads, D, 4)
    what = f"workspace of trees, D={D} heads={heads} group={group} max_q={max_q}"
    step(what)
    want = call(c, max_q)
    space = room(need)
    got = call(c, max_q, ws=space[:need])
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 0, what
    assert (space[need:] == 0x5A).all(), what
    for a, b in zip(got, want):
        assert torch.equal(a, b), what


def test_select_past_4_gib():
    """1024 lists of a table of more than 2^20 places: the keys of the last lists lie past 4 GiB."""
    seqs, heads, page, keep = 128, 8, 64, 2000
    kv = [0] * seqs
    kv[0], kv[5], kv[126], kv[127] = 2100, 2000, 33000, 2001
    c = select_case(kv, heads, page, seed=3, positions=True)
    wide = torch.full((seqs, (1 << 20) // page + 1), -1, dtype=torch.int32, device=DEV)
    wide[:, :c["table"].shape[1]] = c["table"]
    c["table"] = wide
    need = nv.nvfp4_workspace_size(nv._lib.OP_KV_SELECT, 0, 0, heads, wide.shape[1] * page, seqs)
    assert need > 2 * (1 << 32)
    step("selection past 4 GiB")
    space = room(need)
    moves, lens = nv.nvfp4_kv_select(c["w"], c["table"], c["kv_lens"], page, keep, positions=c["pos"],
                                     next_positions=c["nxt"], sinks=4, recent=300, ws=space[:need])
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 0
    assert (space[need:] == 0x5A).all()
    want, want_lens = chosen(c["w"], c["pos"], c["table"], c["kv_lens"], page, keep, c["nxt"], 4, 300, moves.shape[2])
    assert (moves[[0, 126, 127]] >= 0).any(2).all()
    np.testing.assert_array_equal(lens.cpu().numpy(), want_lens)
    np.testing.assert_array_equal(moves.cpu().numpy(), want)
