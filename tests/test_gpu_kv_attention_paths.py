"""GPU parity of nvfp4_kv_attention's launches that short sequences in narrow tables do not reach: shares of
the tokens joined by a second launch, tiles of many rows and their splits, and any of them for any max_q."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from precision_moe_gemm_amd import _lib
from tests.attn_check import assert_attention
from tests.gpu_util import step
from tests.test_gpu_kv_attention import DEV, EDGES, call, check, make_case, reference

pytestmark = pytest.mark.gpu


def widen(c, tokens):
    """The same sequences in a table of at least `tokens` tokens per row, the new entries no pages."""
    t = c["table"]
    wide = torch.full((t.shape[0], max(t.shape[1], -(-tokens // c["page"]))), -1, dtype=torch.int32, device=DEV)
    wide[:, :t.shape[1]] = t
    c["table"] = wide
    return c


# ---- shares -------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (1, 16), (2, 3), (3, 2), (4, 8), (8, 4), (5, 32), (4, 20)])
def test_shares(D, heads, group):
    c = make_case([1] * len(EDGES), EDGES, heads, group, D, 16, seed=D + heads, decode=True)
    check(widen(c, 1040), f"shares D={D} heads={heads} group={group}")


@pytest.mark.parametrize("page", [16, 32, 48, 64, 112, 256])
def test_shares_pages(page):
    lens = [page - 1, page, page + 1, 3 * page - 5, 2 * page + 16, 1, 1100]
    check(make_case([1] * len(lens), lens, 2, 4, 128, page, seed=page, decode=True), f"shares page={page}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_shares_drafts(D):
    q_lens, kv_lens = [2, 5, 1, 3, 0, 4, 7], [2, 1500, 33, 65, 40, 16, 3]
    check(make_case(q_lens, kv_lens, 2, 4, D, 16, seed=D), f"shares drafts D={D}")
    c = make_case(q_lens, kv_lens, 2, 4, D, 16, seed=D + 1)
    check(c, f"shares drafts window D={D}", window=37)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kvh,group,seqs,m", [(4, 4, 1, 20000), (8, 4, 4, 3000), (2, 20, 3, 2000), (1, 1, 12, 1500),
                                              (16, 2, 40, 200), (3, 30, 20, 150)])
def test_joins(D, kvh, group, seqs, m):
    """Few tiles of many parts, many of few: every split of the joining launch's waves."""
    r = np.random.default_rng(seqs)
    lens = [int(v) for v in r.integers(m // 2, m, seqs)]
    check(widen(make_case([1] * seqs, lens, kvh, group, D, 16, seed=m, decode=True), 1040), f"joins {D} {kvh} {group} {m}")


@pytest.mark.parametrize("seqs", [64, 65, 129, 5000])
def test_many_sequences(seqs):
    r = np.random.default_rng(seqs)
    q_lens, kv_lens = [int(v) for v in r.integers(0, 3, seqs)], [int(v) for v in r.integers(0, 40, seqs)]
    c = make_case(q_lens, kv_lens, 1, 2, 64, 16, seed=seqs)
    check(c, f"{seqs} sequences")
    check(widen(c, 1040), f"{seqs} sequences, shares")
    c["max_q"] = 1000
    check(c, f"{seqs} sequences, tiles")


# ---- tiles ---------------------------------------------------------------------
# (rows of the longest sequence times group: 40, then 128 and more)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group,most", [(1, 1, 40), (2, 1, 65), (2, 2, 64), (3, 1, 129), (1, 5, 70), (4, 8, 17), (1, 40, 4)])
@pytest.mark.parametrize("page", [16, 48])
def test_tiles(D, heads, group, most, page):
    q_lens = [most, 1, 0, most - 1, 3]
    kv_lens = [most, 200, 64, most + 63, 2]
    check(make_case(q_lens, kv_lens, heads, group, D, page, seed=D + most), f"tiles {D} {heads} {group} {most} {page}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("most", [50, 150])
def test_tiles_lengths(D, most):
    """Contexts that end in, at and behind a block of 64 tokens and its pages."""
    kv_lens = [most, most + 13, 191, 192, 193, 255, 256, 257, 320]
    kv_lens = [max(v, most) for v in kv_lens]
    check(make_case([most] + [2, most // 2] * 4, kv_lens, 1, 2, D, 32, seed=D + most), f"tiles lengths {D} {most}")


@pytest.mark.parametrize("D,rows", [(64, 40), (64, 100), (64, 200), (128, 40), (128, 100), (128, 200), (256, 70)])
@pytest.mark.parametrize("page", [16, 112, 256])
def test_tiles_split(D, rows, page):
    """Few tiles on a long context: its tokens are split over workgroups and joined."""
    c = make_case([rows, 1], [2900, 1], 1, 1, D, page, seed=rows + page)
    check(c, f"split {D} {rows} {page}")
    if page == 16:
        check(c, f"split {D} {rows} not causal", causal=False)
        check(c, f"split {D} {rows} window", window=700)
        check(c, f"split {D} {rows} short window", window=5)


@pytest.mark.parametrize("most", [60, 200])
def test_tiles_windows(most):
    for window in (1, 31, 64, 65, 128, 4000):
        c = make_case([most, 6, 3], [most + 300, 77, 2], 2, 2, 128, 16, seed=window)
        check(c, f"tiles window={window} {most}", window=window)
    check(c, f"tiles {most} not causal", causal=False)


def test_tiles_pages_before_the_window_may_be_gone():
    c = make_case([150, 140], [700, 300], 2, 2, 64, 16, seed=8)
    whole, _ = call(c, window=50)
    c["table"][0, :(551 - 50) // 16] = -1
    c["table"][1, :(161 - 50) // 16] = 1 << 30
    check(c, "tiles window with freed pages", window=50)
    again, _ = call(c, window=50)
    assert torch.equal(whole, again)


def test_tiles_bad_pages():
    for most in (20, 60, 150):  # rows, 128-row and 256-row tiles
        c = make_case([most, 2], [400, 70], 2, 2, 128, 16, seed=most)
        c["table"][0, 3] = -5
        c["table"][0, 16] = 1 << 28
        c["table"][1, 0] = (1 << 31) - 1
        step(f"bad pages {most}")
        out, lse = call(c)
        torch.cuda.synchronize()
        assert nv.nvfp4_get_error() == _lib.RANGE
        assert_attention(out, lse, reference(c), f"bad pages {most}")
        assert nv.nvfp4_get_error() == 0


def test_tiles_rows_without_keys():
    for most in (50, 150):
        c = make_case([most, 70, 3, 5], [4, 10, 0, 5], 2, 2, 128, 16, seed=21)
        check(c, f"rows without keys {most}")
        check(c, f"rows without keys {most}, not causal", causal=False)


@pytest.mark.parametrize("q_lens", [[9, 2], [60, 2], [150, 2]])
def test_largest_window(q_lens):
    """The largest window there is, on rows before position 0 too."""
    c = make_case(q_lens, [5, 40], 2, 2, 64, 16, seed=22)
    want, _ = call(c)
    check(c, f"window 2^31 - 1, {q_lens}", window=2 ** 31 - 1)
    got, _ = call(c, window=2 ** 31 - 1)
    assert torch.equal(got, want)


# ---- any launch for any call -----------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
def test_any_max_q(D):
    """max_q chooses the launch, never the result."""
    c = make_case([1, 70, 0, 3], [1300, 100, 9, 3], 2, 3, D, 16, seed=D)
    ref = reference(c)
    for max_q in (0, 1, 5, 6, 10, 11, 40, 43, 74, 10 ** 6):
        c["max_q"] = max_q
        step(f"max_q={max_q} D={D}")
        out, lse = call(c)
        torch.cuda.synchronize()
        assert nv.nvfp4_get_error() == 0
        assert_attention(out, lse, ref, f"max_q={max_q}")


def test_more_units_than_31_bits():
    """2000 rows and room for 2^26 tokens in the table: too many units for the row kernel."""
    c = make_case([2000], [2100], 1, 16, 64, 16, seed=7)
    c["max_q"] = 1
    check(widen(c, 1 << 26), "31 bits")


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [50, 2, 9], [200, 2, 9]])
def test_offsets_that_go_down_write_nothing(q_lens):
    c = make_case(q_lens, [300, 40, 30], 2, 2, 64, 16, seed=53)
    n = sum(q_lens)
    for cu in ([0, n, 0, n], [0, n, n - 1, n], [0, -7, 5, n], [n, 0, 0, 0], [2 ** 31 - 1, -2 ** 31, 0, n]):
        c["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        for wide in (False, True):
            d = widen(dict(c), 1100) if wide else c
            out, lse = torch.full_like(c["q"], 7.0), torch.full(c["q"].shape[:2], 7.0, device=DEV)
            step(f"offsets {cu} {wide}")
            call(d, out=out, lse=lse)
            torch.cuda.synchronize()
            assert nv.nvfp4_get_error() == _lib.RANGE
            assert (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 3], [70, 40]), ([1, 3], [1500, 40]), ([60, 3], [70, 40]),
                                            ([200, 3], [300, 40])])
def test_a_row_with_nan_spoils_itself_alone(q_lens, kv_lens):
    c = make_case(q_lens, kv_lens, 2, 2, 128, 16, seed=3)
    want, want_lse = call(c)
    for value in (float("nan"), float("inf"), -float("inf")):
        c["q"] = c["q"].clone()
        c["q"][0, 1, 5], c["q"][-1, 3, 120] = value, value
        step(f"{value} in q")
        out, lse = call(c)
        same = torch.ones(want.shape[:2], dtype=torch.bool, device=DEV)
        same[0, 1], same[-1, 3] = False, False
        assert torch.equal(out[same], want[same]) and torch.equal(lse[same], want_lse[same])
        assert out[0, 1].isnan().any() and out[-1, 3].isnan().any() and not lse[~same].isfinite().any()


CALLS = [([1] * 5, [1500, 30, 1, 0, 700], "shares"), ([1] * 5, [90, 30, 1, 0, 64], "one launch"),
         ([15, 2, 0, 9, 5], [1500, 30, 1, 50, 70], "shares of 32 rows"), ([60, 2, 0, 30, 5], [900, 30, 1, 50, 70], "128-row tiles"), ([200, 2, 0, 30, 5], [2500, 30, 1, 50, 70], "split")]


@pytest.mark.parametrize("q_lens,kv_lens,what", CALLS)
def test_workspace_is_enough_and_may_hold_anything(q_lens, kv_lens, what):
    c = make_case(q_lens, kv_lens, 2, 2, 64, 16, seed=4)
    want, want_lse = call(c)
    n, qh, D = c["q"].shape
    need = nv.nvfp4_workspace_size(_lib.OP_KV_ATTENTION, n, qh, 2, D, len(kv_lens))
    for fill in (0xFF, 0x7F, 0):
        buf = torch.full((need + 512,), fill, dtype=torch.uint8, device=DEV)
        step(f"workspace of {fill}, {what}")
        out, lse = call(c, ws=buf[:need])
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert (buf[need:] == fill).all()
    with pytest.raises(nv.NVFP4Error):
        call(c, ws=buf[:need - 1])


@pytest.mark.parametrize("seqs,group", [(100, 70), (128, 65), (60, 129), (3, 100)])
def test_workspace_of_single_tokens_of_wide_groups(seqs, group):
    """Tiles of many rows without cu_q: what is counted exactly and what the workspace was sized for."""
    c = widen(make_case([1] * seqs, [int(v) for v in np.random.default_rng(1).integers(1, 60, seqs)], 1, group, 64, 16,
                        seed=group, decode=True), 4096)
    need = nv.nvfp4_workspace_size(_lib.OP_KV_ATTENTION, seqs, group, 1, 64, seqs)
    buf = torch.full((need + (1 << 22),), 0xFF, dtype=torch.uint8, device=DEV)
    step(f"single tokens of {seqs} sequences, group {group}")
    out, lse = call(c, ws=buf[:need])
    torch.cuda.synchronize()
    assert (buf[need:] == 0xFF).all()
    assert_attention(out, lse, reference(c), f"single tokens, group {group}")


@pytest.mark.parametrize("q_lens,kv_lens,what", CALLS)
def test_graph_replays(q_lens, kv_lens, what):
    """Captured once; lengths, pages and offsets are read at every replay."""
    c = make_case(q_lens, kv_lens, 2, 4, 128, 16, seed=5)
    full, pages, cu = c["kv_lens"].clone(), c["table"].clone(), c["cu_q"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(c)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    step(f"capture {what}")
    with torch.cuda.graph(graph):
        out, lse = call(c)
    for rep, cut in enumerate((0, 3, 20, 0)):
        c["kv_lens"].copy_((full - cut).clamp(min=0))
        c["table"].copy_(pages if rep < 2 else torch.where(pages >= 0, pages.flip(0).clamp(min=0), 0))
        c["cu_q"].copy_((cu - rep).clamp(min=0))
        out.fill_(5.0)
        want, want_lse = torch.full_like(out, 5.0), torch.full_like(lse, 5.0)
        call(c, out=want, lse=want_lse)
        lse.fill_(5.0)
        torch.cuda.synchronize()
        step(f"replay {rep} {what}")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), rep
    assert nv.nvfp4_get_error() in (0, _lib.RANGE)


def test_two_streams_at_once():
    """Calls of every launch on two streams, each with its own workspace."""
    cases = [make_case(q, m, 2, 4, 128, 16, seed=6) for q, m, _ in CALLS]
    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    step("two streams")
    for rep in range(8):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[(i + rep) % 2]):
                got.append((i, call(c)))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_checks_see_the_queries_and_not_the_unwritten_pages():
    c = make_case([1, 2], [40, 20], 2, 2, 64, 16, seed=9)
    old = nv.nvfp4_set_checks(True)
    try:
        call(c)  # (pages that no sequence holds have NaN scales)
        assert nv.nvfp4_get_error() == 0
        c["q"][1, 0, 3] = float("nan")
        call(c)
        assert nv.nvfp4_get_error() == _lib.DATA
    finally:
        nv.nvfp4_set_checks(old)


def test_tables_of_strided_rows_and_overlapping_ones():
    c = make_case([1, 1, 1], [100, 33, 64], 2, 2, 64, 16, seed=10, decode=True)
    want, _ = call(c)
    wide = torch.full((3, 40), 1 << 30, dtype=torch.int32, device=DEV)
    wide[:, 5:5 + c["table"].shape[1]] = c["table"]
    t = c["table"]
    c["table"] = wide[:, 5:5 + t.shape[1]]
    got, _ = call(c)
    assert torch.equal(got, want)
    c["table"] = t[:1].expand(3, -1)
    with pytest.raises(ValueError):
        call(c)
    c["table"] = t
    with pytest.raises(ValueError):
        call(c, ws=torch.empty(1 << 28, dtype=torch.uint8))
