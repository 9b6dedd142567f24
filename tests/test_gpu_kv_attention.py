"""GPU parity: attention over the paged NVFP4 cache against its formula in 64 bits.

Bounds are those of attn_check.attention, derived from the roundings that the header documents."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.attn_check import assert_attention, attention
from tests.gpu_util import step

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make_cache(pool, page, heads, D, seed, spread=1.0):
    """Two cache tensors of `pool` pages with keys and values of unequal channels, and spare memory
    around them that no kernel may turn into output: every unwritten byte is 0xFF."""
    g = torch.Generator().manual_seed(seed)
    caches = []
    for _ in range(2):
        x = (torch.randn((pool * page * heads, D), generator=g) * torch.exp(
            spread * torch.randn(D, generator=g))).bfloat16()
        t = nv.nvfp4_quantize(x.to(DEV)) if pool else nv.NVFP4Tensor.empty(0, D, 1, DEV)
        caches.append(t)
    return caches


def make_case(q_lens, kv_lens, heads, group, D, page, seed=0, spare=3, spread=1.0, qscale=1.0, decode=False):
    g = torch.Generator().manual_seed(seed + 100)
    need = [-(-m // page) for m in kv_lens]
    pool = sum(need) + spare
    kc, vc = make_cache(pool, page, heads, D, seed, spread)
    order = torch.randperm(pool, generator=g).int()
    table = torch.full((len(kv_lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    # what no sequence owns must not matter: NaN scale bytes and all-ones codes there and behind each end
    own = torch.zeros((pool, page), dtype=torch.bool)
    for b, m in enumerate(kv_lens):
        for p in range(need[b]):
            own[table[b, p], :min(page, m - p * page)] = True
    for t in (kc, vc):
        t.packed.view(pool, page, -1)[~own.to(DEV)] = 0xFF
        t.scales.view(pool, page, -1)[~own.to(DEV)] = 0x7F
    n = sum(q_lens)
    q = (qscale * torch.randn((n, heads * group, D), generator=g)).bfloat16().to(DEV)
    cu = None if decode else torch.tensor(np.r_[0, np.cumsum(q_lens)], dtype=torch.int32, device=DEV)
    return dict(q=q, k_cache=kc, v_cache=vc, heads=heads, table=table.to(DEV),
                kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=DEV), page=page, cu_q=cu,
                max_q=max(q_lens))


def call(c, **kw):
    return nv.nvfp4_kv_attention(c["q"], c["k_cache"], c["v_cache"], c["heads"], c["table"], c["kv_lens"], c["page"],
                                 cu_q=c["cu_q"], max_q=c["max_q"], return_lse=True, **kw)


def reference(c, **kw):
    return attention(c["q"], c["k_cache"], c["v_cache"], c["heads"], c["table"], c["kv_lens"], c["page"],
                     cu_q=c["cu_q"], **kw)


def check(c, what, **kw):
    step(what)
    out, lse = call(c, **kw)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 0, what
    assert_attention(out, lse, reference(c, **kw), what)


# ---- single tokens ---------------------------------------------------------
EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 129, 200, 0]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (1, 16), (2, 3), (3, 2), (4, 8), (8, 4), (5, 1)])
def test_decode_lengths(D, heads, group):
    c = make_case([1] * len(EDGES), EDGES, heads, group, D, 16, seed=D + heads, decode=True)
    check(c, f"decode D={D} heads={heads} group={group}")


@pytest.mark.parametrize("page", [16, 32, 48, 64, 112, 256])
def test_decode_pages(page):
    lens = [page - 1, page, page + 1, 3 * page - 5, 2 * page + 16, 1]
    c = make_case([1] * len(lens), lens, 2, 4, 128, page, seed=page, decode=True)
    check(c, f"decode page={page}")


def test_decode_one_sequence_of_each_length():
    for m in (1, 16, 33, 700, 3001):
        check(make_case([1], [m], 4, 4, 128, 16, seed=m, decode=True), f"decode one sequence of {m}")


@pytest.mark.parametrize("group", [5, 16, 17, 24, 32, 40, 64])
def test_decode_wide_groups(group):
    check(make_case([1] * 3, [70, 1, 133], 2, group, 64, 16, seed=group, decode=True), f"decode group={group}")


def test_decode_many_sequences():
    r = np.random.default_rng(3)
    lens = [int(v) for v in r.integers(0, 80, 700)]
    check(make_case([1] * 700, lens, 1, 2, 64, 16, seed=9, decode=True), "decode 700 sequences")


def test_decode_long_ragged():
    lens = [9000, 3, 0, 517, 1, 4095, 64]
    check(make_case([1] * len(lens), lens, 2, 4, 64, 32, seed=4, decode=True), "decode long ragged")


# ---- several tokens ----------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 4), (2, 3), (4, 2), (3, 1)])
def test_draft_tokens(D, heads, group):
    q_lens, kv_lens = [2, 5, 1, 3, 0, 4], [2, 100, 33, 65, 40, 16]
    check(make_case(q_lens, kv_lens, heads, group, D, 16, seed=D), f"draft D={D} heads={heads} group={group}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts(D):
    q_lens, kv_lens = [1, 17, 64, 65, 130, 33], [1, 17, 64, 65, 130, 33]
    check(make_case(q_lens, kv_lens, 2, 4, D, 16, seed=D), f"prompts D={D}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_on_a_context(D, causal):
    q_lens, kv_lens = [70, 128, 1, 40], [333, 129, 500, 41]
    check(make_case(q_lens, kv_lens, 1, 5, D, 32, seed=D + causal), f"chunks D={D} causal={causal}", causal=causal)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 33, 100, 4000])
def test_windows(window):
    c = make_case([1, 6, 90, 0, 200], [300, 77, 90, 50, 260], 2, 2, 64, 16, seed=window)
    check(c, f"window={window}", window=window)
    d = make_case([1] * 4, [300, 1, 64, 129], 2, 2, 128, 16, seed=window, decode=True)
    check(d, f"decode window={window}", window=window)


def test_pages_before_the_window_may_be_gone():
    c = make_case([1, 40], [300, 200], 2, 2, 64, 16, seed=8)
    whole, _ = call(c, window=50)
    c["table"][0, :(300 - 50) // 16] = -1
    c["table"][1, :(161 - 50) // 16] = 1 << 30
    check(c, "window with freed pages", window=50)
    again, _ = call(c, window=50)
    assert torch.equal(whole, again)


def test_rows_without_keys():
    """More query rows than cached tokens: the rows at positions before 0 see nothing."""
    c = make_case([9, 70, 3, 5], [4, 10, 0, 5], 2, 2, 128, 16, seed=21)
    check(c, "rows without keys")
    out, lse = call(c)
    assert (out[:5] == 0).all() and torch.isinf(lse[:5]).all()
    check(c, "rows without keys, not causal", causal=False)


def test_sharp_and_flat_scores():
    """Scores far apart, alike, and all equal."""
    for qscale in (40.0, 1e-3, 0.0):
        c = make_case([1, 20], [500, 300], 2, 4, 128, 16, seed=5, qscale=qscale)
        check(c, f"scores of queries x {qscale}")


def test_a_growing_maximum():
    """Keys whose scores rise along the sequence: the running maximum grows at every step."""
    c = make_case([1, 33], [600, 600], 1, 4, 64, 16, seed=6)
    x = torch.linspace(-6, 6, 600)[:, None] * torch.ones(64)
    qk = nv.nvfp4_quantize(x.bfloat16().to(DEV))
    c["k_cache"].global_.copy_(qk.global_)
    for b in range(2):
        for p in range(38):
            m = min(16, 600 - 16 * p)
            at = int(c["table"][b, p]) * 16
            c["k_cache"].packed[0, at:at + m] = qk.packed[0, 16 * p:16 * p + m]
            c["k_cache"].scales[0, at:at + m] = qk.scales[0, 16 * p:16 * p + m]
    c["q"] = c["q"].abs()
    check(c, "rising scores")
    c["q"] = -c["q"]
    check(c, "falling scores")


def test_queries_of_unequal_size():
    """Elements of one row spread over 2^40: q is held relative to its row's largest."""
    c = make_case([1, 9], [90, 64], 2, 2, 64, 16, seed=13)
    e = torch.randint(-30, 10, c["q"].shape, generator=torch.Generator().manual_seed(1)).to(DEV)
    c["q"] = torch.ldexp(c["q"].float(), e).bfloat16()
    check(c, "queries of unequal size", scale=1e-3)


def test_strided_rows_and_rows_behind_the_last_sequence():
    c = make_case([3, 20], [40, 90], 2, 2, 128, 16, seed=17)
    n, qh, D = c["q"].shape
    wide = torch.randn((n + 5, qh * D + 136), device=DEV).bfloat16()
    wide[:n, 8:8 + qh * D] = c["q"].reshape(n, -1)
    plain, plain_lse = call(c)
    c["q"] = wide[:, 8:8 + qh * D].unflatten(1, (qh, D))
    outw = torch.full((n + 5, qh * D + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n + 5, qh), 7.0, device=DEV)
    step("strided rows")
    out, _ = call(c, out=outw[:, 16:16 + qh * D].unflatten(1, (qh, D)), lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out[:n], plain) and torch.equal(lse[:n], plain_lse)
    assert (outw[n:] == 7).all() and (lse[n:] == 7).all()
    assert (outw[:, :16] == 7).all() and (outw[:, 16 + qh * D:] == 7).all()


def test_shared_pages():
    """Two sequences with a common prefix in the same pages give what copies of the pages give."""
    c = make_case([1, 1], [64, 64], 2, 2, 128, 16, seed=31, decode=True)
    c["table"][1, :3] = c["table"][0, :3]
    check(c, "shared pages")


def test_same_call_twice_is_the_same():
    c = make_case([1] * 5, [5000, 40, 1, 0, 700], 4, 4, 128, 16, seed=41, decode=True)
    a, la = call(c)
    for _ in range(3):
        b, lb = call(c)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_bad_pages_and_lengths_raise_and_stay_in_bounds():
    c = make_case([1, 1, 20], [100, 64, 50], 2, 2, 64, 16, seed=51)
    c["table"][0, 2] = -5
    c["table"][2, 1] = 1 << 28
    step("bad pages")
    out, lse = call(c)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 3
    assert_attention(out, lse, reference(c), "bad pages are skipped")
    # a length past the table is cut, a negative one is none
    d = make_case([1, 1], [112, 30], 2, 2, 64, 16, seed=52, decode=True)
    want, _ = call(d)
    d["kv_lens"] = torch.tensor([2000, -3], dtype=torch.int32, device=DEV)
    step("bad lengths")
    got, _ = call(d)
    assert nv.nvfp4_get_error() == 3
    assert torch.equal(got[0], want[0]) and (got[1] == 0).all()
    # query offsets outside [0, n]
    e = make_case([2, 3], [40, 30], 2, 2, 64, 16, seed=53)
    e["cu_q"] = torch.tensor([0, 2, 900], dtype=torch.int32, device=DEV)
    step("bad offsets")
    call(e)
    assert nv.nvfp4_get_error() == 3
    e["cu_q"] = torch.tensor([0, -7, 5], dtype=torch.int32, device=DEV)
    call(e)
    assert nv.nvfp4_get_error() == 3
    assert nv.nvfp4_get_error() == 0


def test_nothing_to_do():
    c = make_case([1, 2], [20, 20], 2, 2, 64, 16, seed=61)
    q0 = c["q"][:0]
    out = nv.nvfp4_kv_attention(q0, c["k_cache"], c["v_cache"], 2, c["table"], c["kv_lens"], 16,
                                cu_q=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert out.shape == q0.shape
    none = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    out = torch.full_like(c["q"], 3.0)
    nv.nvfp4_kv_attention(c["q"], c["k_cache"], c["v_cache"], 2, none, none[:, 0], 16,
                          cu_q=torch.zeros(1, dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    assert (out == 3).all()


def test_offsets_past_32_bits():
    """A cache whose codes pass 4 GiB: pages at its far end."""
    heads, D, page = 4, 256, 64
    c = make_case([1, 20], [150, 200], heads, 2, D, page, seed=71)
    small = c["k_cache"].rows // heads // page
    pool = (5 << 30) // (page * heads * D // 2)
    for name in ("k_cache", "v_cache"):
        s = c[name]
        big = nv.NVFP4Tensor.empty(pool * page * heads, D, 1, DEV)
        big.packed[0, -s.rows:] = s.packed[0]
        big.scales[0, -s.rows:] = s.scales[0]
        big.global_.copy_(s.global_)
        c[name + "_small"], c[name] = s, big
    want = attention(c["q"], c["k_cache_small"], c["v_cache_small"], heads, c["table"], c["kv_lens"], page,
                     cu_q=c["cu_q"])
    c["table"] = torch.where(c["table"] >= 0, c["table"] + (pool - small), -1).int()
    step("offsets past 32 bits")
    out, lse = call(c)
    torch.cuda.synchronize()
    assert_attention(out, lse, want, "offsets past 32 bits")


def test_another_stream_and_graph_replays():
    """Captured once, replayed while the sequences grow: every replay equals the eager call."""
    c = make_case([1] * 4, [400, 90, 33, 250], 2, 4, 128, 16, seed=81, decode=True)
    full = c["kv_lens"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = call(c)
    torch.cuda.current_stream().wait_stream(side)
    assert_attention(out, lse, reference(c), "another stream")
    step("graph capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call(c)
    for rep, cut in enumerate((0, 7, 30, 1)):
        c["kv_lens"].copy_((full - cut).clamp(min=0))
        eager, eager_lse = call(c)
        out.zero_()
        torch.cuda.synchronize()
        step(f"graph replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, eager_lse), rep


def test_refusals_of_the_binding():
    c = make_case([1, 1], [20, 20], 2, 2, 64, 16, seed=91, decode=True)
    args = [c["q"], c["k_cache"], c["v_cache"], 2, c["table"], c["kv_lens"], 16]

    def bad(i, v, exc, **kw):
        a = list(args)
        a[i] = v
        with pytest.raises(exc):
            nv.nvfp4_kv_attention(*a, **kw)

    bad(0, c["q"].float(), ValueError)
    bad(0, c["q"][..., :32], ValueError)
    bad(0, c["q"].transpose(1, 2).contiguous().transpose(1, 2), ValueError)
    bad(0, c["q"].cpu(), ValueError)
    bad(3, 3, nv.NVFP4Error)
    bad(4, c["table"].long(), ValueError)
    bad(5, c["kv_lens"][:1], ValueError)
    bad(6, 24, nv.NVFP4Error)
    bad(6, 0, nv.NVFP4Error)
    bad(0, c["q"], nv.NVFP4Error, scale=float("nan"))
    bad(0, c["q"], nv.NVFP4Error, scale=-1.0)
    bad(0, c["q"], nv.NVFP4Error, causal=False, window=3)
    bad(0, c["q"], ValueError, cu_q=torch.zeros(2, dtype=torch.int32, device=DEV))
    bad(0, c["q"], ValueError, out=torch.empty((2, 4, 32), dtype=torch.bfloat16, device=DEV))
