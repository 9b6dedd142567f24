"""GPU parity: the attention weight that cached tokens receive, against its formula in 64 bits.

Bounds are those of cache_check.received, derived from the roundings of the kernels."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.cache_check import received
from tests.gpu_util import step
from tests.test_gpu_kv_attention import make_case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(q_lens, kv_lens, heads, group, D, page, seed=0, **kw):
    c = make_case(q_lens, kv_lens, heads, group, D, page, seed=seed, **kw)
    g = torch.Generator().manual_seed(seed + 7)
    tokens = c["k_cache"].rows // heads
    c["before"] = torch.exp(2 * torch.randn((heads, tokens), generator=g)).to(DEV)
    return c


def with_lse(c, **kw):
    _, c["lse"] = nv.nvfp4_kv_attention(c["q"], c["k_cache"], c["v_cache"], c["heads"], c["table"], c["kv_lens"], c["page"],
                                        cu_q=c["cu_q"], max_q=c["max_q"], return_lse=True, **kw)
    return c


def call(c, out=None, weights="before", max_q=None, **kw):
    before = c["before"] if isinstance(weights, str) else weights
    out = torch.full_like(c["before"], 7.0) if out is None else out
    return nv.nvfp4_kv_weights(c["q"], c["lse"], c["k_cache"], c["heads"], c["table"], c["kv_lens"], c["page"], out,
                               weights=before, cu_q=c["cu_q"], max_q=c["max_q"] if max_q is None else max_q, **kw)


def agree(got, ref, rest, what):
    """rest: what the tokens of no sequence hold."""
    want, tol, written = ref
    got = got.cpu().double()
    d = (got - want).abs()
    bad = written & ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(d[written].max()), [int(v) for v in bad.nonzero()[0]],
                           float(got[bad][0]), float(want[bad][0]), float(tol[bad][0]))
    rest = rest.cpu().double().expand_as(got) if isinstance(rest, torch.Tensor) else torch.full_like(got, rest)
    assert torch.equal(got[~written], rest[~written]), (what, "tokens of no sequence")


def check(c, what, max_q=None, **kw):
    step(what)
    if "lse" not in c:
        with_lse(c, **kw)
    out = call(c, max_q=max_q, **kw)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 0, what
    args = (c["q"], c["lse"], c["k_cache"], c["heads"], c["table"], c["kv_lens"], c["page"])
    ref = received(*args, c["before"], cu_q=c["cu_q"], **kw)
    agree(out, ref, 7.0, what)
    # in place
    mine = c["before"].clone()
    call(c, out=mine, weights=mine, max_q=max_q, **kw)
    torch.cuda.synchronize()
    written = ref[2]
    if not kw.get("window"):
        assert torch.equal(mine.cpu()[written], out.cpu()[written]), what
    agree(mine, ref, c["before"], what + ", in place")
    return out


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 129, 600, 0]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (4, 8), (8, 4), (5, 1), (1, 16), (2, 32)])
def test_single_tokens(D, heads, group):
    check(make([1] * len(EDGES), EDGES, heads, group, D, 16, seed=D + heads, decode=True),
          f"weights D={D} heads={heads} group={group}")


@pytest.mark.parametrize("page", [16, 32, 48, 64, 112, 256])
def test_pages(page):
    lens = [page - 1, page, page + 1, 3 * page - 5, 2 * page + 16, 1]
    check(make([1] * len(lens), lens, 2, 4, 128, page, seed=page, decode=True), f"page={page}")
    check(make(lens, lens, 2, 2, 128, page, seed=page), f"prompts, page={page}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_and_many_sequences(D):
    """Runs longer than what a wave keeps, sequences that end inside a share."""
    check(make([1] * 7, [9000, 3, 0, 517, 1, 4095, 64], 2, 4, D, 32, seed=4, decode=True), f"long ragged D={D}")


def test_700_sequences():
    lens = [int(v) for v in np.random.default_rng(3).integers(0, 80, 700)]
    check(make([1] * 700, lens, 1, 2, 64, 16, seed=9, decode=True), "700 sequences")
    r = np.random.default_rng(5)
    q = [int(v) for v in r.integers(0, 30, 200)]
    check(make(q, [a + int(v) for a, v in zip(q, r.integers(0, 90, 200))], 1, 2, 64, 16, seed=9), "200 chunks")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 4), (2, 3), (3, 1), (1, 33), (1, 40)])
def test_several_rows(D, heads, group):
    q, kv = [2, 5, 1, 3, 0, 4], [2, 100, 33, 65, 40, 16]
    check(make(q, kv, heads, group, D, 16, seed=D), f"several rows D={D} heads={heads} group={group}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts(D):
    q = [1, 17, 64, 65, 130, 33, 300]
    check(make(q, q, 2, 4, D, 16, seed=D), f"prompts D={D}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_on_a_context(D, causal):
    check(make([70, 128, 1, 40], [333, 129, 500, 41], 1, 5, D, 32, seed=D + causal), f"chunks D={D} causal={causal}",
          causal=causal)


@pytest.mark.parametrize("D", [64, 256])
def test_many_rows(D):
    """More rows of a sequence than their shifts' space in shared memory holds (1024 at a time)."""
    check(make([700, 40], [760, 300], 1, 7, D, 16, seed=2), f"many rows D={D}")


@pytest.mark.parametrize("max_q", [1, 4, 8, 200])
def test_max_q_chooses_the_kernel_and_not_the_result(max_q):
    check(make([1, 9, 40, 3], [50, 1100, 700, 3], 2, 4, 128, 16, seed=max_q), f"max_q={max_q}", max_q=max_q)


@pytest.mark.parametrize("max_q", [1, 200])
@pytest.mark.parametrize("window", [1, 2, 16, 31, 33, 100, 4000])
def test_windows(window, max_q):
    c = make([1, 6, 90, 0, 200], [300, 77, 90, 50, 260], 2, 2, 64, 16, seed=window)
    check(c, f"window={window} max_q={max_q}", max_q=max_q, window=window)


@pytest.mark.parametrize("max_q", [1, 200])
def test_rows_without_keys(max_q):
    """More query rows than cached tokens: their lse is -inf, and all tokens are their own."""
    c = make([9, 70, 3, 5], [4, 10, 0, 5], 2, 2, 128, 16, seed=21)
    check(c, "rows without keys", max_q=max_q)
    del c["lse"]
    check(c, "rows without keys, not causal", max_q=max_q, causal=False)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tiles_of_many_sequences(D):
    """More sequences than a wave has lanes, blocks that are and are not split."""
    r = np.random.default_rng(D)
    q = [int(v) for v in r.integers(0, 30, 90)]
    c = make(q, [a + int(v) for a, v in zip(q, r.integers(0, 300, 90))], 1, 3, D, 16, seed=D)
    check(c, f"90 sequences in tiles D={D}", max_q=200)
    check(make([1] * 300, [int(v) for v in r.integers(1, 600, 300)], 4, 2, D, 16, seed=D), f"300 sequences D={D}", max_q=200)


@pytest.mark.parametrize("max_q", [1, 16, 200])
def test_many_heads(max_q):
    check(make([2, 7], [40, 70], 268, 1, 64, 16, seed=5), f"268 KV heads max_q={max_q}", max_q=max_q)
    check(make([2, 7], [40, 70], 129, 2, 64, 16, seed=5), f"129 KV heads max_q={max_q}", max_q=max_q)


@pytest.mark.parametrize("max_q", [1, 32, 200])
def test_the_widest_window(max_q):
    c = make([3, 40], [90, 300], 2, 2, 128, 16, seed=37)
    check(c, f"window=2^31-1 max_q={max_q}", max_q=max_q, window=2 ** 31 - 1)


@pytest.mark.parametrize("max_q", [0, 200])
def test_no_query_rows_at_all(max_q):
    """The weights are copied, with no query row in the call."""
    c = make([0, 0], [90, 33], 2, 2, 64, 16, seed=35)
    c["lse"] = torch.empty((0, 4), device=DEV)
    step(f"no query rows max_q={max_q}")
    out = call(c, max_q=max_q)
    mine = c["before"].clone()
    call(c, out=mine, weights=mine, max_q=max_q)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 0
    assert torch.equal(mine, c["before"])
    own = torch.zeros_like(out, dtype=torch.bool)
    for b, kv in enumerate((90, 33)):
        t = torch.arange(kv, device=DEV)
        own[:, c["table"][b].long()[t // 16] * 16 + t % 16] = True
    assert torch.equal(out, torch.where(own, c["before"], 7.0))


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [40, 1, 9]])
def test_the_sum_over_all_tokens_is_the_number_of_rows(q_lens):
    """No weights before: what a KV head's tokens receive adds up to its rows."""
    c = with_lse(make(q_lens, [900, 30, 77], 2, 4, 128, 16, seed=12))
    out = call(c, out=torch.zeros_like(c["before"]), weights=None)
    torch.cuda.synchronize()
    want = torch.full((2,), 4.0 * sum(q_lens), dtype=torch.float64)
    assert torch.allclose(out.cpu().double().sum(1), want, rtol=1e-4)


def test_no_weights_before_and_sequences_without_rows():
    c = with_lse(make([0, 3, 0], [200, 90, 33], 2, 2, 64, 16, seed=33))
    step("no weights before")
    out = call(c, weights=None)
    ref = received(c["q"], c["lse"], c["k_cache"], 2, c["table"], c["kv_lens"], 16, None, cu_q=c["cu_q"])
    agree(out, ref, 7.0, "no weights before")
    slot = c["table"][0, :12].long().cpu()[:, None] * 16 + torch.arange(16)
    assert (out.cpu()[:, slot.flatten()] == 0).all()  # no row: nothing received


@pytest.mark.parametrize("max_q", [1, 200])
def test_rows_that_count_for_nothing(max_q):
    """NaN and infinities in q, and an lse that is none."""
    c = with_lse(make([6, 40], [90, 300], 2, 2, 128, 16, seed=41))
    c["q"][1, 0, 3] = float("nan")
    c["q"][20, 3, 100] = float("inf")
    c["q"][21, 1, 0] = -float("inf")
    c["lse"][3, 1] = float("nan")
    c["lse"][4, 2] = float("inf")
    c["lse"][30, 0] = -float("inf")
    step("rows that count for nothing")
    out = call(c, max_q=max_q)
    torch.cuda.synchronize()
    ref = received(c["q"], c["lse"], c["k_cache"], 2, c["table"], c["kv_lens"], 16, c["before"], cu_q=c["cu_q"])
    # (a row with an infinity adds nothing here, and 0 or 1 where its score is infinite: two rows, one a KV head)
    want, tol, written = ref
    got = out.cpu().double()
    assert torch.isfinite(got[written]).all()
    assert ((got - want) >= -tol)[written].all()
    assert ((got - want) <= tol + 1)[written].all()
    own = torch.zeros_like(written)  # the first sequence has no such row
    t = torch.arange(90)
    own[:, c["table"][0].cpu().long()[t // 16] * 16 + t % 16] = True
    assert ((got - want).abs() <= tol)[own].all()


def test_a_weight_is_at_most_one():
    """Log-sum-exps that are not those of the rows."""
    c = with_lse(make([1, 30], [90, 200], 2, 2, 64, 16, seed=43))
    c["lse"] -= 300.0  # (not what the attention gave: every weight would be huge)
    for max_q in (1, 200):
        out = call(c, weights=None, out=torch.zeros_like(c["before"]), max_q=max_q)
        torch.cuda.synchronize()
        assert (out >= 0).all() and (out <= 60).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("max_q", [1, 200])
def test_bad_pages_lengths_and_offsets(max_q):
    c = with_lse(make([1, 1, 20], [100, 64, 50], 2, 2, 64, 16, seed=51))
    c["table"][0, 2] = -5
    c["table"][2, 1] = 1 << 28
    step("bad pages")
    out = call(c, max_q=max_q)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 3
    agree(out, received(c["q"], c["lse"], c["k_cache"], 2, c["table"], c["kv_lens"], 16, c["before"], cu_q=c["cu_q"]), 7.0,
          "bad pages are skipped")
    d = with_lse(make([1, 1], [112, 30], 2, 2, 64, 16, seed=52, decode=True))
    want = call(d, max_q=max_q)
    d["kv_lens"] = torch.tensor([2000, -3], dtype=torch.int32, device=DEV)
    step("bad lengths")
    got = call(d, max_q=max_q)
    assert nv.nvfp4_get_error() == 3
    slot = (d["table"][0].long()[:, None] * 16 + torch.arange(16, device=DEV)).flatten()
    assert torch.equal(got[:, slot], want[:, slot])
    e = with_lse(make([2, 3], [40, 30], 2, 2, 64, 16, seed=53))
    for offsets in ([0, 2, 900], [0, -7, 5]):
        e["cu_q"] = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        step(f"bad offsets {offsets}")
        call(e, max_q=max_q)
        assert nv.nvfp4_get_error() == 3
    assert nv.nvfp4_get_error() == 0


@pytest.mark.parametrize("max_q", [1, 200])
def test_strided_weights_and_queries(max_q):
    c = with_lse(make([3, 20], [40, 90], 2, 2, 128, 16, seed=17))
    plain = call(c, max_q=max_q)
    n, qh, D = c["q"].shape
    tokens = c["before"].shape[1]
    wide = torch.randn((n, qh * D + 136), device=DEV).bfloat16()
    wide[:, 8:8 + qh * D] = c["q"].reshape(n, -1)
    c["q"] = wide[:, 8:8 + qh * D].unflatten(1, (qh, D))
    both = torch.full((2, 2 * tokens + 5), 7.0, device=DEV)
    both[:, 1:1 + tokens] = c["before"]
    c["before"] = both[:, 1:1 + tokens]
    step("strided weights")
    out = call(c, out=both[:, tokens + 3:2 * tokens + 3], max_q=max_q)
    torch.cuda.synchronize()
    assert torch.equal(out, plain)
    assert (both[:, 0] == 7).all() and (both[:, tokens + 1:tokens + 3] == 7).all() and (both[:, -2:] == 7).all()


def test_same_call_twice_and_graph_replays():
    """In a graph with its own workspace, replayed while the sequences grow; weights add up over the replays."""
    need = nv.nvfp4_workspace_size(nv._lib.OP_KV_WEIGHTS, 30, 8, 2, 128, 4)
    for c, what in ((make([1] * 4, [400, 90, 33, 250], 2, 4, 128, 16, seed=81, decode=True), "single tokens"),
                    (make([20, 3, 7, 0], [400, 90, 33, 250], 2, 4, 128, 16, seed=82), "chunks")):
        with_lse(c)
        a = call(c)
        for _ in range(3):
            assert torch.equal(call(c), a)
        full, mine = c["kv_lens"].clone(), c["before"].clone()
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        step(f"graph capture, {what}")
        with torch.cuda.graph(graph):
            call(c, out=mine, weights=mine, ws=ws)
        mine.copy_(c["before"])
        eager = c["before"].clone()
        for rep, cut in enumerate((0, 7, 30, 1)):
            c["kv_lens"].copy_((full - cut).clamp(min=0))
            call(c, out=eager, weights=eager)
            torch.cuda.synchronize()
            step(f"graph replay {rep}")
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(mine, eager), (what, rep)


def test_another_stream():
    c = with_lse(make([30, 2], [90, 400], 2, 4, 128, 16, seed=83))
    want = call(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(c)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_offsets_past_32_bits():
    """A cache whose codes pass 4 GiB: pages at its far end."""
    heads, D, page = 4, 256, 64
    for q_lens in ([1, 1], [1, 60]):
        c = with_lse(make(q_lens, [150, 200], heads, 2, D, page, seed=71))
        small, s = c["k_cache"].rows // heads // page, c["k_cache"]
        want, tol, written = received(c["q"], c["lse"], s, heads, c["table"], c["kv_lens"], page, c["before"], cu_q=c["cu_q"])
        pool = (5 << 30) // (page * heads * D // 2)
        big = nv.NVFP4Tensor.empty(pool * page * heads, D, 1, DEV)
        big.packed[0, -s.rows:] = s.packed[0]
        big.scales[0, -s.rows:] = s.scales[0]
        big.global_.copy_(s.global_)
        before = torch.zeros((heads, pool * page), device=DEV)
        before[:, -small * page:] = c["before"]
        c["k_cache"], c["before"] = big, before
        c["table"] = torch.where(c["table"] >= 0, c["table"] + (pool - small), -1).int()
        step("offsets past 32 bits")
        out = call(c)
        torch.cuda.synchronize()
        assert nv.nvfp4_get_error() == 0
        agree(out[:, -small * page:], (want, tol, written), 7.0, "offsets past 32 bits")


def test_refusals_of_the_binding():
    c = with_lse(make([2, 3], [20, 20], 2, 2, 64, 16, seed=91))
    out = torch.zeros_like(c["before"])

    def bad(exc, **kw):
        with pytest.raises(exc):
            nv.nvfp4_kv_weights(**dict(dict(q=c["q"], lse=c["lse"], k_cache=c["k_cache"], heads=2, block_table=c["table"],
                                            kv_lens=c["kv_lens"], page_size=16, out=out, weights=c["before"],
                                            cu_q=c["cu_q"]), **kw))

    bad(ValueError, q=c["q"].float())
    bad(ValueError, lse=c["lse"][:2])
    bad(ValueError, lse=c["lse"].double())
    bad(ValueError, out=out[:, :-1])
    bad(ValueError, out=out[:1])
    bad(ValueError, out=out.double())
    bad(ValueError, weights=c["before"].cpu())
    bad(ValueError, weights=c["before"][:1].expand(2, -1))
    store = torch.zeros(3 * out.shape[1], device=DEV)
    bad(nv.NVFP4Error, weights=store[:2 * out.shape[1]].view(2, -1), out=store[1:1 + 2 * out.shape[1]].view(2, -1))
    bad(nv.NVFP4Error, page_size=24)
    bad(nv.NVFP4Error, scale=0.0)
    bad(nv.NVFP4Error, causal=False, window=3)
    bad(ValueError, cu_q=c["cu_q"][:2])
