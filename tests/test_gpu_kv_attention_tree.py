"""GPU parity: attention of trees of drafts over the paged NVFP4 cache against its formula in 64 bits.

Bounds are those of attn_check.attention, derived from the roundings that the header documents."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.attn_check import assert_attention
from tests.cache_check import bits_of, mask_of, tree_attention
from tests.gpu_util import step
from tests.test_gpu_kv_attention import make_case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def trees(q_lens, r, words=None):
    """Ancestor masks of random trees, all sequences' rows one under the other."""
    widest = max(max(q_lens), 1)
    bits = np.zeros((sum(q_lens), 32 * (-(-widest // 32) if words is None else words)), dtype=bool)
    at = 0
    for m in q_lens:
        for i in range(m):
            parent = int(r.integers(-1, i)) if i else -1
            if parent >= 0:
                bits[at + i] = bits[at + parent]
            if i < bits.shape[1]:
                bits[at + i, i] = True
        at += m
    return bits


def make(q_lens, kv_lens, heads, group, D, page, seed=0, bits=None, **kw):
    c = make_case(q_lens, kv_lens, heads, group, D, page, seed=seed, **kw)
    c["mask"] = mask_of(trees(q_lens, np.random.default_rng(seed)) if bits is None else bits).to(DEV)
    return c


def call(c, max_q=None, **kw):
    return nv.nvfp4_kv_attention_tree(c["q"], c["k_cache"], c["v_cache"], c["heads"], c["table"], c["kv_lens"], c["page"],
                                      c["cu_q"], c["mask"], max_q=c["max_q"] if max_q is None else max_q,
                                      return_lse=True, **kw)


def reference(c, **kw):
    return tree_attention(c["q"], c["k_cache"], c["v_cache"], c["heads"], c["table"], c["kv_lens"], c["page"], c["cu_q"],
                          c["mask"], **kw)


def widened(c):
    """The same sequences in rows of the table of more than 1024 tokens (which take other launches)."""
    more = torch.full((c["table"].shape[0], -(-1025 // c["page"])), -1, dtype=torch.int32, device=DEV)
    return dict(c, table=torch.cat([c["table"], more], 1))


def check(c, what, max_q=None, **kw):
    want = reference(c, **kw)
    results = []
    for x, table in ((c, "its own table"), (widened(c), "a wide table")):
        step(f"{what}, {table}")
        out, lse = call(x, max_q, **kw)
        torch.cuda.synchronize()
        assert nv.nvfp4_get_error() == 0, (what, table)
        assert_attention(out, lse, want, f"{what}, {table}")
        results.append((out, lse))
    return results[0]


# contexts that end inside and at the end of pages, of steps of 32 and of blocks of 64; trees of one word, of
# exactly one, of several; no context at all
M = [1, 2, 7, 31, 32, 33, 64, 65, 0, 40]
KV = [1, 33, 7, 40, 64, 100, 128, 300, 20, 200]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (4, 2), (1, 8)])
def test_trees(D, heads, group):
    check(make(M, KV, heads, group, D, 16, seed=D + heads), f"trees D={D} heads={heads} group={group}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("m", [1, 3, 8, 16])
def test_small_trees_on_short_and_long_contexts(D, m):
    """Row tiles: a launch of whole tiles (tables of up to 1024 tokens), and shares with a joining launch."""
    check(make([m] * 3, [m + 500, m, m + 63], 2, 4, D, 16, seed=m), f"small trees of {m} D={D}")
    check(make([m] * 3, [m + 1500, m, m + 63], 2, 4, D, 48, seed=m), f"small trees of {m} on 1500 D={D}")


@pytest.mark.parametrize("max_q", [1, 4, 20, 200])
def test_max_q_chooses_the_kernel_and_not_the_result(max_q):
    check(make([1, 9, 40, 3], [50, 1100, 700, 3], 2, 4, 128, 16, seed=max_q), f"max_q={max_q}", max_q=max_q)
    check(make([1, 9, 40, 3], [50, 1100, 700, 3], 2, 4, 64, 16, seed=max_q), f"max_q={max_q}, heads of 64", max_q=max_q)


@pytest.mark.parametrize("page", [16, 32, 48, 112, 256])
def test_pages(page):
    m = [5, 20, 33, 9]
    check(make(m, [page + 2, page, 3 * page - 5, 2 * page + 9], 2, 4, 128, page, seed=page), f"page={page}")


@pytest.mark.parametrize("D,max_q", [(64, 8), (64, 40), (128, 8), (128, 40), (128, 130), (256, 8), (256, 130)])
@pytest.mark.parametrize("window", [1, 2, 5, 31, 33, 100, 4000])
def test_windows(window, D, max_q):
    """The last `window` of what a row sees, drafts among them: windows below, at and above a path's length."""
    c = make([40, 7, 20, 3], [300, 77, 20, 90], 2, 2, D, 16, seed=window)
    check(c, f"window={window} D={D} max_q={max_q}", max_q=max_q, window=window)


@pytest.mark.parametrize("max_q", [2, 12, 100])
@pytest.mark.parametrize("window", [0, 9])
def test_any_bits(max_q, window):
    """Rows of random bits, of none, of all, and bits of drafts that do not exist."""
    r = np.random.default_rng(5)
    m = [9, 33, 2, 70]
    bits = r.random((sum(m), 96)) < 0.4
    bits[3] = bits[20] = bits[42] = bits[80] = False
    bits[30] = bits[50] = True
    c = make(m, [200, 33, 2, 1200], 2, 2, 128, 16, seed=6, bits=bits)
    out, lse = check(c, f"any bits max_q={max_q} window={window}", max_q=max_q, window=window)
    assert (out[20] == 0).all() and torch.isinf(lse[20]).all()  # nothing before the drafts, and no draft
    # the same without the bits behind each tree, in rows apart from each other
    at = 0
    for k in m:
        bits[at:at + k, k:] = False
        at += k
    wide = torch.full((sum(m), 11), -1, dtype=torch.int32, device=DEV)
    wide[:, 4:7] = mask_of(bits).to(DEV)
    c["mask"] = wide[:, 4:7]
    again, _ = call(c, max_q, window=window)
    assert torch.equal(out, again)


def test_a_chain_is_what_the_causal_attention_gives():
    c = make([5, 1, 30], [300, 64, 90], 2, 4, 128, 16, seed=9, bits=np.tril(np.ones((36, 32), dtype=bool)))
    rows = [np.tril(np.ones((m, 32), dtype=bool)) for m in (5, 1, 30)]
    c["mask"] = mask_of(np.concatenate(rows)).to(DEV)
    for window in (0, 3, 50):
        out, lse = check(c, f"chain window={window}", window=window)
        want, want_lse = nv.nvfp4_kv_attention(c["q"], c["k_cache"], c["v_cache"], 2, c["table"], c["kv_lens"], 16,
                                               cu_q=c["cu_q"], max_q=30, window=window, return_lse=True)
        assert (out.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
        assert (lse - want_lse).abs().max() < 1e-4


def test_single_drafts_without_offsets():
    c = make([1] * 5, [1, 16, 40, 0, 33], 2, 4, 128, 16, seed=3, decode=True)
    assert c["cu_q"] is None
    check(c, "single drafts")
    c["mask"].zero_()  # they do not even see themselves
    out, _ = check(c, "single drafts that see the context alone")
    assert (out[0] == 0).all()


def test_fewer_cached_tokens_than_drafts():
    """The first drafts are not cached: they are seen by nobody."""
    for window in (0, 2):
        c = make([9, 70, 3, 5], [4, 10, 0, 5], 2, 2, 128, 16, seed=21)
        check(c, f"more drafts than tokens, window={window}", window=window)


@pytest.mark.parametrize("table", [dict, widened])
@pytest.mark.parametrize("max_q", [2, 100])
def test_too_few_words(max_q, table):
    """Drafts behind the mask's words raise an error and are hidden."""
    c = table(make([40, 20], [140, 60], 2, 2, 128, 16, seed=4))
    bits = bits_of(c["mask"])[:, :32]
    c["mask"] = mask_of(bits).to(DEV)
    step("too few words")
    out, lse = call(c, max_q)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 3 and nv.nvfp4_get_error() == 0
    assert_attention(out, lse, reference(c), "too few words")
    c["mask"] = c["mask"][:, :0]  # none at all: the tokens before the drafts
    out, lse = call(c, max_q)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 3
    assert_attention(out, lse, reference(c), "no words")


@pytest.mark.parametrize("table", [dict, widened])
@pytest.mark.parametrize("max_q", [20, 40])
def test_bad_pages_and_pages_before_the_window(max_q, table):
    c = table(make([6, 40], [300, 200], 2, 2, 64, 16, seed=8))
    whole, _ = call(c, max_q, window=50)
    c["table"][0, :(300 - 6 - 50) // 16] = -1
    c["table"][1, :(200 - 40 - 50) // 16] = 1 << 30
    out, _ = check(c, "window with freed pages", max_q, window=50)
    assert torch.equal(whole, out)
    c["table"][0, 18] = -7  # the drafts' page
    step("bad page")
    out, lse = call(c, max_q, window=50)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 3
    assert_attention(out, lse, reference(c, window=50), "a bad page is skipped")


@pytest.mark.parametrize("table", [dict, widened])
@pytest.mark.parametrize("max_q", [20, 200])
def test_strided_rows_and_rows_behind_the_last_sequence(max_q, table):
    c = table(make([3, 20], [40, 90], 2, 2, 128, 16, seed=17))
    n, qh, D = c["q"].shape
    plain, plain_lse = call(c, max_q)
    wide = torch.randn((n + 5, qh * D + 136), device=DEV).bfloat16()
    wide[:n, 8:8 + qh * D] = c["q"].reshape(n, -1)
    c["q"] = wide[:, 8:8 + qh * D].unflatten(1, (qh, D))
    c["mask"] = torch.cat([c["mask"], torch.full((5, 1), -1, dtype=torch.int32, device=DEV)])
    outw = torch.full((n + 5, qh * D + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n + 5, qh), 7.0, device=DEV)
    step("strided rows")
    out, _ = call(c, max_q, out=outw[:, 16:16 + qh * D].unflatten(1, (qh, D)), lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out[:n], plain) and torch.equal(lse[:n], plain_lse)
    assert (outw[n:] == 7).all() and (lse[n:] == 7).all()
    assert (outw[:, :16] == 7).all() and (outw[:, 16 + qh * D:] == 7).all()


@pytest.mark.parametrize("table", [dict, widened])
@pytest.mark.parametrize("max_q", [4, 60])
def test_a_row_of_nan_spoils_itself_alone(max_q, table):
    c = table(make([20, 9], [90, 400], 2, 2, 128, 16, seed=23))
    want, want_lse = call(c, max_q)
    c["q"][5, 1, 7] = float("nan")
    out, lse = call(c, max_q)
    torch.cuda.synchronize()
    assert torch.isnan(out[5, 1]).all()
    out[5, 1], lse[5, 1] = want[5, 1], want_lse[5, 1]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_many_sequences():
    r = np.random.default_rng(3)
    m = [int(v) for v in r.integers(0, 12, 300)]
    kv = [a + int(v) for a, v in zip(m, r.integers(0, 60, 300))]
    check(make(m, kv, 1, 2, 64, 16, seed=9), "300 sequences")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_q", [40, 200])
def test_tiles_of_many_sequences(D, max_q):
    """Shares of the tile kernel that hold many tiles, of more sequences than a wave has lanes."""
    r = np.random.default_rng(D)
    m = [int(v) for v in r.integers(0, 40, 90)]
    kv = [a + int(v) for a, v in zip(m, r.integers(0, 400, 90))]
    check(make(m, kv, 1, 3, D, 16, seed=D), f"90 trees D={D} max_q={max_q}", max_q=max_q)
    check(make(m[:20], kv[:20], 2, 9, D, 16, seed=D), f"20 trees, several tiles each, D={D}", max_q=max_q)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tiles_of_many_shares(D):
    """A long context beside short ones: a tile that many workgroups share."""
    c = make([33, 2, 40], [20000, 100, 3000], 1, 8, D, 64, seed=D)
    check(c, f"long beside short D={D}")
    check(c, f"long beside short D={D}, window", window=2500)


@pytest.mark.parametrize("max_q", [4, 20, 70, 200])
def test_many_heads(max_q):
    check(make([3, 40], [90, 130], 268, 1, 64, 16, seed=4), f"268 KV heads max_q={max_q}", max_q=max_q)
    check(make([3, 40], [90, 130], 515, 1, 64, 16, seed=4), f"515 KV heads max_q={max_q}", max_q=max_q)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_short_contexts_by_the_number_of_trees(D):
    """Tables of up to 1024 tokens: tiles of 16 rows, of 32, and shares."""
    for seqs in (1, 3, 8, 12):
        kv = [100 + 61 * b for b in range(seqs)]
        check(make([16] * seqs, kv, 8, 4, D, 16, seed=seqs), f"{seqs} trees of 16 D={D}")


@pytest.mark.parametrize("max_q", [8, 20, 200])
def test_the_widest_window(max_q):
    check(make([9, 40], [90, 300], 2, 2, 128, 16, seed=37), f"window=2^31-1 max_q={max_q}", max_q=max_q, window=2 ** 31 - 1)


@pytest.mark.parametrize("table", [dict, widened])
def test_another_stream_graph_replays_and_a_workspace_each(table):
    """Two captured graphs with a workspace each, replayed while contexts and masks change."""
    c = table(make([9, 3, 20], [400, 90, 633], 2, 4, 128, 16, seed=81))
    full, bits = c["kv_lens"].clone(), bits_of(c["mask"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = call(c)
    torch.cuda.current_stream().wait_stream(side)
    assert_attention(out, lse, reference(c), "another stream")
    need = nv.nvfp4_workspace_size(nv._lib.OP_KV_ATTENTION_TREE, 32, 8, 2, 128, 3)
    graphs = []
    for max_q in (9, 40):
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        step(f"graph capture max_q={max_q}")
        with torch.cuda.graph(graph):
            got = call(c, max_q, ws=ws)
        graphs.append((graph, max_q, *got))
    for rep, cut in enumerate((0, 7, 30, 1)):
        c["kv_lens"].copy_((full - cut).clamp(min=0))
        c["mask"].copy_(mask_of(np.roll(bits, rep, axis=1)))
        eager = [call(c, g[1]) for g in graphs]
        torch.cuda.synchronize()
        step(f"graph replay {rep}")
        for g in graphs:
            g[2].zero_()
            g[0].replay()
        torch.cuda.synchronize()
        for g, (o, z) in zip(graphs, eager):
            assert torch.equal(g[2], o) and torch.equal(g[3], z), rep


def test_refusals_of_the_binding():
    c = make([2, 3], [20, 20], 2, 2, 64, 16, seed=91)

    def bad(exc, **kw):
        with pytest.raises(exc):
            nv.nvfp4_kv_attention_tree(**dict(dict(q=c["q"], k_cache=c["k_cache"], v_cache=c["v_cache"], heads=2,
                                                   block_table=c["table"], kv_lens=c["kv_lens"], page_size=16,
                                                   cu_q=c["cu_q"], mask=c["mask"]), **kw))

    bad(ValueError, mask=c["mask"].long())
    bad(ValueError, mask=c["mask"][:3])
    bad(ValueError, mask=c["mask"].cpu())
    bad(ValueError, mask=c["mask"].expand(5, 4))
    bad(nv.NVFP4Error, window=-1)
    bad(nv.NVFP4Error, scale=0.0)
    bad(ValueError, cu_q=c["cu_q"][:2])
