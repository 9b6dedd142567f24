"""GPU parity: received weights in place under a window, whose earlier pages a sequence may have given up.

What a call leaves alone is compared in its bits: it holds -0.0, which adding nothing would turn into 0.0."""
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.cache_check import received
from tests.gpu_util import step
from tests.test_gpu_kv_weights import DEV, agree, make, with_lse

pytestmark = pytest.mark.gpu


def in_place(c, table, max_q, **kw):
    w = c["before"].clone()
    nv.nvfp4_kv_weights(c["q"], c["lse"], c["k_cache"], c["heads"], table, c["kv_lens"], c["page"], w, weights=w,
                        cu_q=c["cu_q"], max_q=max_q, **kw)
    torch.cuda.synchronize()
    return w


def places(c, b, t0, t1):
    t = torch.arange(t0, t1, device=DEV)
    return c["table"][b].long()[t // c["page"]] * c["page"] + t % c["page"]


def bits(t):
    return t.view(torch.int32)


# rows and tokens of each sequence: windows that begin in a page, at its first token, in the first step or block of
# tokens and in later ones
Q, KV = [1, 6, 90, 1, 200, 2], [300, 77, 620, 1040, 260, 40]


@pytest.mark.parametrize("max_q", [1, 16, 32, 200])
@pytest.mark.parametrize("D,heads,group,page", [(64, 2, 2, 16), (128, 2, 2, 16), (256, 1, 2, 16), (128, 1, 3, 48),
                                                (64, 268, 1, 16), (256, 140, 1, 32)])
def test_pages_given_up_before_the_window(D, heads, group, page, max_q):
    """(With many heads the tile kernel's blocks are not split over their rows, else they are.)"""
    window = 50
    c = with_lse(make(Q, KV, heads, group, D, page, seed=D + page), window=window)
    first = [max(0, kv - q - window + 1) for q, kv in zip(Q, KV)]
    for b, lo in enumerate(first):
        c["before"][:, places(c, b, 0, lo)] = -0.0
    what = f"D={D} heads={heads} page={page} max_q={max_q}"
    step(f"window, {what}")
    want = in_place(c, c["table"], max_q, window=window)
    assert nv.nvfp4_get_error() == 0, what
    ref = list(received(c["q"], c["lse"], c["k_cache"], heads, c["table"], c["kv_lens"], page, c["before"], cu_q=c["cu_q"],
                        window=window))
    for b, lo in enumerate(first):
        ref[2][:, places(c, b, 0, lo).cpu()] = False
    agree(want, ref, c["before"], what)
    assert torch.equal(bits(want)[~ref[2].to(DEV)], bits(c["before"])[~ref[2].to(DEV)]), what
    pool = c["k_cache"].rows // heads // page
    held = [c["table"][b, :-(-kv // page)] for b, kv in enumerate(KV)]
    for kind in ("none", "past the cache", "of the sequence itself", "of the next sequence"):
        table = c["table"].clone()
        for b, lo in enumerate(first):
            gone = lo // page
            other = held[(b + 1) % len(KV)] if kind == "of the next sequence" else held[b].flip(0)
            table[b, :gone] = (torch.full((gone,), -1 if kind == "none" else pool, dtype=torch.int32, device=DEV)
                               if kind in ("none", "past the cache") else other.repeat(gone)[:gone])
        step(f"window, entries before it: {kind}, {what}")
        got = in_place(c, table, max_q, window=window)
        assert nv.nvfp4_get_error() == 0, (kind, what)
        assert torch.equal(bits(got), bits(want)), (kind, what)


@pytest.mark.parametrize("max_q", [1, 16, 32, 200])
@pytest.mark.parametrize("window", [0, 40])
def test_sequences_without_rows_are_left_alone(window, max_q):
    """Idle slots, whose rows of the table may hold anything, beside others and with no other."""
    for q, kv in (([0, 3, 0, 0, 1], [200, 90, 33, 64, 300]), ([0, 0], [95, 600])):
        c = make(q, kv, 2, 2, 128, 16, seed=6)
        with_lse(c, window=window) if sum(q) else c.update(lse=torch.empty((0, 4), device=DEV))
        idle = [b for b in range(len(q)) if q[b] == 0]
        for b in idle:
            c["before"][:, places(c, b, 0, kv[b])] = -0.0
        what = f"idle slots {idle}, window={window} max_q={max_q}"
        step(what)
        want = in_place(c, c["table"], max_q, window=window)
        assert nv.nvfp4_get_error() == 0, what
        ref = list(received(c["q"], c["lse"], c["k_cache"], 2, c["table"], c["kv_lens"], 16, c["before"], cu_q=c["cu_q"],
                            window=window))
        for b in idle:
            ref[2][:, places(c, b, 0, kv[b]).cpu()] = False
        agree(want, ref, c["before"], what)
        assert torch.equal(bits(want)[~ref[2].to(DEV)], bits(c["before"])[~ref[2].to(DEV)]), what
        for entry in (-1, 1 << 24, "another's"):
            table = c["table"].clone()
            for b in idle:
                other = c["table"][(b + 1) % len(q)]
                table[b] = other.clamp(min=0) if entry == "another's" else entry
            step(f"{what}, entries {entry}")
            got = in_place(c, table, max_q, window=window)
            assert nv.nvfp4_get_error() == 0, (entry, what)
            assert torch.equal(bits(got), bits(want)), (entry, what)


@pytest.mark.parametrize("max_q", [1, 200])
def test_a_bad_page_in_the_window_is_reported(max_q):
    c = with_lse(make([1, 3], [300, 200], 2, 2, 64, 16, seed=3), window=40)
    for entry in (-1, 1 << 20):
        table = c["table"].clone()
        table[0, 261 // 16] = entry  # (the window begins at token 260)
        step(f"a bad page in the window, {entry}")
        got = in_place(c, table, max_q, window=40)
        assert nv.nvfp4_get_error() == 3
        assert torch.equal(got[:, places(c, 0, 256, 272)], c["before"][:, places(c, 0, 256, 272)])
    assert nv.nvfp4_get_error() == 0
