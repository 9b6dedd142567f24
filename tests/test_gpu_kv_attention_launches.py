"""GPU: nvfp4_kv_attention's tile launches where only max_q or the table's width leads to them, each shown to be the
one that ran by what it leaves in the workspace: a tile launch that does not split leaves it alone, one that does
begins it with a record of its number of tiles, as the row launch with shares does."""
import pytest
import torch

import precision_moe_gemm_amd as nv
from precision_moe_gemm_amd import _lib
from tests.attn_check import assert_attention, attention
from tests.gpu_util import step
from tests.test_gpu_kv_attention import DEV, call, make_case, reference
from tests.test_gpu_kv_attention_paths import widen

pytestmark = pytest.mark.gpu


def run(c, what, ref, **kw):
    """The call against ref; the number of tiles in the workspace's second word, None where nothing was written."""
    n, qh, D = c["q"].shape
    need = nv.nvfp4_workspace_size(_lib.OP_KV_ATTENTION, n, qh, c["heads"], D, len(c["kv_lens"]))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    step(what)
    out, lse = call(c, ws=ws, **kw)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 0
    assert_attention(out, lse, ref, what)
    return None if bool((ws == 0xFF).all()) else int(ws[4:8].view(torch.int32))


def row_units(rows, per, tokens):
    """Units of the row launch that the host counts for one sequence of `rows` query rows per KV head."""
    return (rows + per - 1) // per * (-(-tokens // 32) + 1)


@pytest.mark.parametrize("q,page,pages,tiles", [(2000, 16, 1 << 23, None), (70, 256, 0x7FFFFF00 // 256, 9)])
def test_too_many_units_for_either_row_tile(q, page, pages, tiles):
    """More than 2^31 - 1 units in tiles of 16 rows (a group of 16) and of 32: the tiles of 128 rows take the call,
    whole (250 of them) or split, in the widest table that there is."""
    assert min(row_units(16 * q, per, page * pages) for per in (16, 32)) > 2 ** 31 - 1
    c = make_case([q], [2100], 1, 16, 64, page, seed=7)
    c["max_q"] = 1
    ref = reference(c)
    assert run(widen(c, page * pages), f"{q} rows, {page * pages} tokens in the table", ref) == tiles


@pytest.mark.parametrize("D,max_q", [(64, 64), (64, 100), (128, 64), (128, 100), (256, 64)])
def test_tiles_past_32_bits(D, max_q):
    """Caches whose codes pass 4 GiB, pages at their far end: tiles of 128 rows (max_q * group up to 128, and heads
    of 256) and of 256."""
    heads, page = 4, 64
    c = make_case([1, 20], [150, 200], heads, 2, D, page, seed=D)
    c["max_q"] = max_q
    ref = reference(c)
    small = c["k_cache"].rows // heads // page
    pool = (5 << 30) // (page * heads * D // 2)
    for name in ("k_cache", "v_cache"):
        s = c[name]
        big = nv.NVFP4Tensor.empty(pool * page * heads, D, 1, DEV)
        big.packed[0, -s.rows:] = s.packed[0]
        big.scales[0, -s.rows:] = s.scales[0]
        big.global_.copy_(s.global_)
        c[name] = big
    c["table"] = torch.where(c["table"] >= 0, c["table"] + (pool - small), -1).int()
    assert run(c, f"tiles past 32 bits, D = {D}, max_q = {max_q}", ref) is None


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 112, 256])
def test_forty_rows_in_split_tiles(D, page):
    c = make_case([40, 1], [2900, 1], 1, 1, D, page, seed=40 + page)
    c["max_q"] = 65
    assert run(c, f"split {D} {page}", reference(c)) == 2
    if page == 16:
        for kw in (dict(causal=False), dict(window=700), dict(window=5)):
            assert run(c, f"split {D} {kw}", reference(c, **kw), **kw) == 2


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 48])
@pytest.mark.parametrize("group,most", [(1, 40), (40, 1), (20, 2)])
def test_forty_rows_in_whole_tiles(D, page, group, most):
    c = make_case([most, 1, 0, most - 1, 3], [most, 200, 64, most + 63, 3], 1, group, D, page, seed=D + most)
    c["max_q"] = 128 // group
    run(c, f"tiles {D} {group} {most} {page}", reference(c))


def test_the_row_launch_begins_its_workspace_with_its_tiles():
    c = widen(make_case([20, 1], [1500, 40], 1, 2, 64, 16, seed=1), 2000)
    assert run(c, "shares", reference(c)) == 3  # tiles of 32 rows: 2 and 1
