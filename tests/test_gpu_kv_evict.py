"""GPU parity: the tokens that a sequence keeps (whole numbers, equal to a plain selection) and moves of cached
tokens (bytes, equal to a plain copy)."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.cache_check import chosen, moved
from tests.gpu_util import step

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---- selection -----------------------------------------------------------------
def make(kv_lens, heads, page, seed=0, positions=False, spare=2, kind="heavy"):
    g = torch.Generator().manual_seed(seed)
    need = [-(-m // page) for m in kv_lens]
    pool = sum(need) + spare
    table = torch.full((len(kv_lens), max(1, max(need))), -1, dtype=torch.int32)
    order, at = torch.randperm(pool, generator=g).int(), 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    shape = (heads, pool * page)
    w = torch.exp(2 * torch.randn(shape, generator=g))
    if kind == "ties":
        w = torch.randint(0, 3, shape, generator=g).float()
    elif kind == "equal":
        w = torch.full(shape, 0.25)
    elif kind == "close":  # neighbours in the last bits
        w = (torch.randint(0, 40, shape, generator=g).int() + 0x3F800000).view(torch.float32)
    elif kind == "odd":
        r = torch.randint(0, 8, shape, generator=g)
        for i, v in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -3.0)):
            w[r == i] = v
    pos = nxt = None
    if positions:
        pos = torch.zeros(shape, dtype=torch.int32)
        nxt = torch.tensor([3 * m + 1 for m in kv_lens], dtype=torch.int32)
        for b, m in enumerate(kv_lens):
            slot = (table[b].long().clamp(min=0)[:, None] * page + torch.arange(page)).flatten()[:m]
            for h in range(heads):
                pos[h, slot] = torch.randperm(3 * m + 1, generator=g)[:m].int()
    return dict(w=w.to(DEV), table=table.to(DEV), kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=DEV), page=page,
                pos=None if pos is None else pos.to(DEV), nxt=None if nxt is None else nxt.to(DEV))


def check(c, keep, sinks=0, recent=0, cap=None, what=""):
    step(f"select keep={keep} sinks={sinks} recent={recent} {what}")
    moves, lens = nv.nvfp4_kv_select(c["w"], c["table"], c["kv_lens"], c["page"], keep, positions=c["pos"],
                                     next_positions=c["nxt"], sinks=sinks, recent=recent, cap=cap)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 0
    want, want_lens = chosen(c["w"], c["pos"], c["table"], c["kv_lens"], c["page"], keep, c["nxt"], sinks, recent,
                             moves.shape[2])
    np.testing.assert_array_equal(lens.cpu().numpy(), want_lens)
    np.testing.assert_array_equal(moves.cpu().numpy(), want)
    return moves


LENS = [1, 16, 17, 63, 64, 65, 100, 1023, 1024, 1025, 2100, 0]


@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "close", "odd"])
@pytest.mark.parametrize("positions", [False, True])
def test_lengths_and_weights(kind, positions):
    c = make(LENS, 3, 16, seed=len(kind), positions=positions, kind=kind)
    for keep, sinks, recent in ((1, 0, 0), (1, 0, 1), (16, 4, 8), (64, 0, 64), (64, 1, 10), (1024, 100, 200), (2099, 3, 7),
                                (2100, 0, 0)):
        check(c, keep, sinks, recent, what=f"{kind} positions={positions}")


@pytest.mark.parametrize("page", [16, 48, 256])
def test_pages(page):
    check(make([page, page + 1, 5 * page - 7], 2, page, seed=page, positions=True), page, 2, 5, what=f"page={page}")


@pytest.mark.parametrize("n", [4095, 4097, 32767, 32769, 70000])
@pytest.mark.parametrize("kind", ["heavy", "ties", "equal"])
def test_long_sequences(n, kind):
    """Around the numbers of keys that shared memory holds, and far past them."""
    c = make([n, n // 3], 2, 64, seed=n, positions=True, kind=kind)
    for keep in (16, n // 2, n - 1):
        check(c, keep, 4 if keep > 20 else 0, min(keep - 4, 300), what=f"{n} tokens, {kind}")


def test_long_and_short_sequences_together():
    """A table of 70000 tokens whose rows are filled by different amounts."""
    for kind in ("heavy", "close", "odd"):
        c = make([70000, 34001, 34000, 33999, 100, 1, 0], 3, 16, seed=9, positions=True, kind=kind)
        for keep, sinks, recent in ((34000, 4, 500), (64, 0, 0), (1, 0, 1), (69999, 5, 0)):
            check(c, keep, sinks, recent, what=f"long and short, {kind}")


def test_long_rows_at_once_and_in_a_graph():
    """A workspace for each of two streams; a graph replayed while lengths and weights change."""
    c, d = make([40000, 33000], 2, 64, seed=1, positions=True), make([50000], 4, 64, seed=2, kind="ties")

    def run(x, ws, keep=9000):
        return nv.nvfp4_kv_select(x["w"], x["table"], x["kv_lens"], x["page"], keep, positions=x["pos"],
                                  next_positions=x["nxt"], sinks=4, recent=300, ws=ws)

    def room(x):
        need = nv.nvfp4_workspace_size(nv._lib.OP_KV_SELECT, 0, 0, x["w"].shape[0], x["table"].shape[1] * x["page"],
                                       x["table"].shape[0])
        return torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)

    want = [run(x, None) for x in (c, d)]
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [room(x) for x in (c, d)]
    torch.cuda.synchronize()
    step("two streams")
    got = []
    for _ in range(3):
        for x, s, ws in zip((c, d), streams, spaces):
            with torch.cuda.stream(s):
                got.append(run(x, ws))
    torch.cuda.synchronize()
    for i, (moves, lens) in enumerate(got):
        assert torch.equal(moves, want[i % 2][0]) and torch.equal(lens, want[i % 2][1]), i
    graph = torch.cuda.CUDAGraph()
    step("graph capture")
    with torch.cuda.graph(graph):
        moves, lens = run(c, spaces[0])
    for rep, now in enumerate(([40000, 33000], [9000, 33000], [39999, 20], [0, 9001])):
        c["kv_lens"].copy_(torch.tensor(now, dtype=torch.int32))
        c["w"].copy_(c["w"].roll(77, 1))
        eager = run(c, None)
        torch.cuda.synchronize()
        step(f"graph replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(moves, eager[0]) and torch.equal(lens, eager[1]), rep
        held = chosen(c["w"], c["pos"], c["table"], c["kv_lens"], c["page"], 9000, c["nxt"], 4, 300, moves.shape[2])
        np.testing.assert_array_equal(moves.cpu().numpy(), held[0])


def test_one_more_token_than_the_budget():
    c = make([129] * 70, 8, 16, seed=3, positions=True)
    moves = check(c, 128, 4, 32)
    assert ((moves[..., 0] >= 0).sum(2) <= 1).all()


def test_more_protected_tokens_than_places():
    """Positions that repeat: of tokens kept first the lowest places stay."""
    c = make([200, 90], 2, 16, seed=5, positions=True)
    c["pos"].fill_(1)
    check(c, 50, 4, 10)
    c["pos"].copy_(torch.randint(0, 6, c["pos"].shape, device=DEV))
    check(c, 50, 4, 10)
    c["nxt"].fill_(-(1 << 31))  # every position counts as recent
    check(c, 50, 0, 50)
    c["nxt"].fill_((1 << 31) - 1)
    c["pos"].fill_((1 << 31) - 1)
    check(c, 50, 0, 50)


@pytest.mark.parametrize("n", [300, 34000])
def test_positions_past_the_newest_count_as_recent(n):
    c = make([n], 2, 16, seed=13, positions=True)
    c["nxt"].fill_(2 * n)  # (positions reach 3 n)
    for recent in (0, 1, 30):
        check(c, n // 2, 0, recent, what="positions past the newest")


def test_strides_and_a_roomy_list():
    c = make([300, 40], 2, 16, seed=7, positions=True)
    wide = torch.full((2, c["w"].shape[1] + 9), float("nan"), device=DEV)
    wide[:, 3:3 + c["w"].shape[1]] = c["w"]
    c["w"] = wide[:, 3:3 + c["w"].shape[1]]
    check(c, 100, 4, 20, cap=250)


def test_bad_pages_and_lengths():
    c = make([300, 100, 60], 2, 16, seed=9)
    c["table"][0, 3], c["table"][0, 7], c["table"][1, 1] = -2, 1 << 20, c["w"].shape[1] // 16
    step("bad pages")
    moves, lens = nv.nvfp4_kv_select(c["w"], c["table"], c["kv_lens"], 16, 80, sinks=2, recent=8)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == 3
    want, _ = chosen(c["w"], None, c["table"], c["kv_lens"], 16, 80, None, 2, 8, moves.shape[2])
    np.testing.assert_array_equal(moves.cpu().numpy(), want)
    d = make([304, 100, 60], 2, 16, seed=10)
    true = chosen(d["w"], None, d["table"], d["kv_lens"], 16, 80, None, 2, 8, 80)[0]
    d["kv_lens"] = torch.tensor([1 << 30, -5, 60], dtype=torch.int32, device=DEV)
    step("bad lengths")
    moves, lens = nv.nvfp4_kv_select(d["w"], d["table"], d["kv_lens"], 16, 80, sinks=2, recent=8)
    assert nv.nvfp4_get_error() == 3
    assert lens.tolist() == [80, 0, 60]
    np.testing.assert_array_equal(moves[0].cpu().numpy(), true[0])
    assert (moves[1:] == -1).all()


# ---- moves ---------------------------------------------------------------------
def cache(pool, page, heads, D, seed):
    g = torch.Generator().manual_seed(seed)
    tensors = []
    for _ in range(2):
        t = nv.NVFP4Tensor.empty(pool * page * heads, D, 1, DEV)
        t.packed.copy_(torch.randint(0, 256, t.packed.shape, generator=g, dtype=torch.uint8))
        t.scales.copy_(torch.randint(0, 256, t.scales.shape, generator=g, dtype=torch.uint8))
        t.global_.fill_(1.0)
        tensors.append(t)
    w = torch.randn((heads, pool * page), generator=g).to(DEV)
    p = torch.randint(0, 1 << 30, (heads, pool * page), generator=g).int().to(DEV)
    return (*tensors, w, p)


def arrays(kc, vc, w, p, heads):
    tokens = kc.rows // heads
    parts = [t.view(tokens, heads, -1).cpu().numpy() for t in (kc.packed, kc.scales, vc.packed, vc.scales)]
    return parts + [w.T.cpu().numpy().copy(), p.T.cpu().numpy().copy()]


def check_move(state, table, page, heads, moves, what, weights=True, positions=True, error=0):
    kc, vc, w, p = state
    want = moved(arrays(kc, vc, w, p, heads), moves, table.cpu().numpy(), page, heads)
    old = arrays(kc, vc, w, p, heads)
    step(what)
    nv.nvfp4_kv_move(kc, vc, heads, table, page, torch.as_tensor(moves, dtype=torch.int32, device=DEV),
                     weights=w if weights else None, positions=p if positions else None)
    torch.cuda.synchronize()
    assert nv.nvfp4_get_error() == error, what
    for i, (got, new, before) in enumerate(zip(arrays(kc, vc, w, p, heads), want, old)):
        keep = (i == 4 and not weights) or (i == 5 and not positions)
        np.testing.assert_array_equal(got, before if keep else new, err_msg=f"{what}, part {i}")


@pytest.mark.parametrize("D", [32, 64, 96, 128, 256, 320, 4096])
@pytest.mark.parametrize("lists", [1, 3])
def test_chains_of_moves(D, lists):
    """Moves whose sources are others' destinations: shifts down and up, a rotation, and any permutation."""
    heads, page, pool = 3, 16, 12
    table = torch.randperm(pool, generator=torch.Generator().manual_seed(D))[:10].view(2, 5).int().to(DEV)
    r = np.random.default_rng(D)
    for cap in (1, 2, 5, 33, 64):
        for kind in ("down", "up", "permutation"):
            moves = np.full((2, lists, cap + (cap > 4), 2), -1, dtype=np.int32)
            for b in range(2):
                for h in range(lists):
                    at = r.permutation(80)[:cap + 1] if kind == "permutation" else np.arange(7, 8 + cap)
                    src, dst = {"down": (at[1:], at[:-1]), "up": (at[:-1], at[1:]),
                                "permutation": (at[:cap], np.roll(at[:cap], 1))}[kind]
                    where = np.sort(r.permutation(moves.shape[2])[:cap])
                    moves[b, h, where, 0], moves[b, h, where, 1] = src, dst
            check_move(cache(pool, page, heads, D, cap), table, page, heads, moves, f"D={D} lists={lists} cap={cap} {kind}")


@pytest.mark.parametrize("cap", [65, 128, 200, 256])
@pytest.mark.parametrize("lists", [1, 2])
def test_permutations_of_up_to_256_tokens(cap, lists):
    heads, page, pool = 2, 32, 20
    r = np.random.default_rng(cap)
    table = torch.randperm(pool, generator=torch.Generator().manual_seed(cap))[:18].view(2, 9).int().to(DEV)
    moves = np.stack([np.stack([np.stack([p, np.roll(p, 1 + b)], 1) for p in (r.permutation(288)[:cap] for _ in range(lists))])
                      for b in range(2)])
    check_move(cache(pool, page, heads, 128, cap), table, page, heads, moves, f"a permutation of {cap}")


@pytest.mark.parametrize("D", [32, 64, 96, 128, 256, 320, 4096])
@pytest.mark.parametrize("lists", [1, 5])
def test_long_lists(D, lists):
    heads, page, pool, cap = 5, 16, 50, 300
    r = np.random.default_rng(D)
    table = torch.randperm(pool, generator=torch.Generator().manual_seed(D))[:48].view(1, 48).int().to(DEV)
    moves = np.full((1, lists, cap, 2), -1, dtype=np.int32)
    for h in range(lists):
        k = cap - 3 * h
        moves[0, h, :k, 0], moves[0, h, :k, 1] = 384 + np.sort(r.permutation(384)[:k]), np.sort(r.permutation(384)[:k])
    check_move(cache(pool, page, heads, D, 1), table, page, heads, moves, f"long lists D={D}")


@pytest.mark.parametrize("cap", [6, 300])
def test_without_weights_or_positions_and_odd_places(cap):
    heads, page, pool = 2, 16, 42
    table = torch.arange(40).view(1, 40).int().to(DEV)
    r = np.random.default_rng(cap)
    moves = np.full((1, 1, cap, 2), -1, dtype=np.int32)
    k = min(cap, 290)
    moves[0, 0, :k, 0], moves[0, 0, :k, 1] = 320 + r.permutation(320)[:k], r.permutation(320)[:k]
    for weights, positions in ((True, False), (False, True), (False, False)):
        check_move(cache(pool, page, heads, 64, 2), table, page, heads, moves, f"{weights} {positions}", weights, positions)
    # places outside the table, a destination before 0, pages that are none
    moves[0, 0, 0], moves[0, 0, 1, 1], moves[0, 0, 2, 0] = (640, 1), -1, (1 << 31) - 1
    moves[0, 0, 3, 0], moves[0, 0, 4, 1] = 17, 40
    table[0, 1], table[0, 2] = -1, 42
    check_move(cache(pool, page, heads, 64, 3), table, page, heads, moves, "odd places", error=3)


def test_nothing_to_move():
    state = cache(3, 16, 2, 64, 1)
    table = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    check_move(state, table, 16, 2, np.zeros((1, 1, 0, 2), dtype=np.int32), "no moves")
    check_move(state, table[:0], 16, 2, np.zeros((0, 1, 4, 2), dtype=np.int32), "no sequences")
    check_move(state, table, 16, 2, np.full((1, 2, 7, 2), -1, dtype=np.int32), "empty lists")
    check_move(state, table, 16, 2, np.array([[[[5, 5]]]], dtype=np.int32), "a token to itself")


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("cap", [5, 40, 200, 300])
def test_one_tensor_as_keys_and_values(D, cap):
    """It is moved once: chains up to 256 moves, else sources that nobody writes."""
    heads, page, pool = 2, 16, 44
    table = torch.randperm(pool, generator=torch.Generator().manual_seed(cap))[:40].view(1, 40).int().to(DEV)
    r = np.random.default_rng(cap)
    moves = np.full((1, heads, cap, 2), -1, dtype=np.int32)
    for h in range(heads):
        at = r.permutation(640)
        moves[0, h, :, 0] = at[:cap]
        moves[0, h, :, 1] = np.roll(at[:cap], 1) if cap <= 256 else at[cap:2 * cap]
    kc, _, w, p = cache(pool, page, heads, D, cap)
    check_move((kc, kc, w, p), table, page, heads, moves, f"K as V, D={D} cap={cap}")


def test_strided_weights():
    kc, vc, w, p = cache(4, 16, 2, 64, 5)
    wide = torch.full((2, 64 + 9), 7.0, device=DEV)
    wide[:, 4:68] = w
    check_move((kc, vc, wide[:, 4:68], p), torch.tensor([[2, 0]], dtype=torch.int32, device=DEV), 16, 2,
               np.array([[[[20, 3], [3, 20]]]], dtype=np.int32), "strided weights")
    assert (wide[:, :4] == 7).all() and (wide[:, 68:] == 7).all()


def test_offsets_past_32_bits():
    heads, D, page = 4, 256, 64
    pool = (5 << 30) // (page * heads * D // 2)
    kc, vc = (nv.NVFP4Tensor.empty(pool * page * heads, D, 1, DEV) for _ in range(2))
    w = torch.zeros((heads, pool * page), device=DEV)
    p = torch.zeros((heads, pool * page), dtype=torch.int32, device=DEV)
    small = cache(6, page, heads, D, 9)
    n = 6 * page
    table = torch.tensor([[pool - 2, pool - 5, pool - 1, pool - 4]], dtype=torch.int32, device=DEV)
    for cap in (100, 300):
        for t, s in ((kc, small[0]), (vc, small[1])):
            t.packed[0, -n * heads:], t.scales[0, -n * heads:] = s.packed[0], s.scales[0]
        w[:, -n:], p[:, -n:] = small[2], small[3]
        r = np.random.default_rng(cap)
        moves = np.full((1, 4, cap, 2), -1, dtype=np.int32)
        for h in range(4):
            moves[0, h, :100, 0], moves[0, h, :100, 1] = 128 + r.permutation(128)[:100], r.permutation(128)[:100]
        want = moved(arrays(*small, heads), moves, (table - (pool - 6)).cpu().numpy(), page, heads)
        step(f"far moves, {cap}")
        nv.nvfp4_kv_move(kc, vc, heads, table, page, torch.from_numpy(moves).to(DEV), weights=w, positions=p)
        torch.cuda.synchronize()
        assert nv.nvfp4_get_error() == 0
        tail = [nv.NVFP4Tensor(t.packed[:, -n * heads:], t.scales[:, -n * heads:], t.global_, n * heads, D) for t in (kc, vc)]
        for got, new in zip(arrays(*tail, w[:, -n:], p[:, -n:], heads), want):
            np.testing.assert_array_equal(got, new)


# ---- both ----------------------------------------------------------------------
def test_selection_and_moves_in_a_graph():
    """Replayed while weights and lengths change: the kept tokens' rows, in the kept order."""
    heads, page, D, keep = 2, 16, 64, 40
    c = make([90, 60, 41, 40, 0], heads, page, seed=11, positions=True)
    pool = c["w"].shape[1] // page
    kc, vc, _, _ = cache(pool, page, heads, D, 3)
    first = [t.clone() for t in (kc.packed, kc.scales, vc.packed, vc.scales, c["w"], c["pos"])]
    now = (kc.packed, kc.scales, vc.packed, vc.scales, c["w"], c["pos"])

    def both():
        moves, lens = nv.nvfp4_kv_select(c["w"], c["table"], c["kv_lens"], page, keep, positions=c["pos"],
                                         next_positions=c["nxt"], sinks=4, recent=8)
        nv.nvfp4_kv_move(kc, vc, heads, c["table"], page, moves, weights=c["w"], positions=c["pos"])
        return moves, lens

    both()
    graph = torch.cuda.CUDAGraph()
    step("graph capture")
    with torch.cuda.graph(graph):
        moves, lens = both()
    for rep in range(4):
        for t, f in zip(now, first):
            t.copy_(f)
        c["w"].mul_(torch.rand(c["w"].shape, device=DEV, generator=torch.Generator(DEV).manual_seed(rep)))
        c["kv_lens"].copy_(torch.tensor([90 - rep, 60, 41 - rep, 40, rep], dtype=torch.int32))
        want, want_lens = chosen(c["w"], c["pos"], c["table"], c["kv_lens"], page, keep, c["nxt"], 4, 8, moves.shape[2])
        rows = moved(arrays(kc, vc, c["w"], c["pos"], heads), want, c["table"].cpu().numpy(), page, heads)
        step(f"graph replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(moves.cpu().numpy(), want)
        np.testing.assert_array_equal(lens.cpu().numpy(), want_lens)
        for got, new in zip(arrays(kc, vc, c["w"], c["pos"], heads), rows):
            np.testing.assert_array_equal(got, new)


def test_refusals_of_the_binding():
    c = make([30], 2, 16, positions=True)
    kc, vc, w, p = cache(4, 16, 2, 64, 5)

    def bad(exc, **kw):
        with pytest.raises(exc):
            nv.nvfp4_kv_select(**dict(dict(weights=c["w"], block_table=c["table"], kv_lens=c["kv_lens"], page_size=16,
                                           keep=20, positions=c["pos"], next_positions=c["nxt"]), **kw))

    bad(ValueError, weights=c["w"].double())
    bad(ValueError, weights=c["w"][0])
    bad(ValueError, positions=c["pos"].long())
    bad(ValueError, positions=c["pos"][:, :-1])
    bad(ValueError, next_positions=None)
    bad(ValueError, next_positions=c["nxt"].repeat(2))
    bad(ValueError, kv_lens=c["kv_lens"].cpu())
    bad(nv.NVFP4Error, keep=0, cap=5)
    bad(nv.NVFP4Error, sinks=15, recent=6)
    bad(nv.NVFP4Error, cap=11)
    bad(nv.NVFP4Error, page_size=24)

    def bad_move(exc, **kw):
        with pytest.raises(exc):
            nv.nvfp4_kv_move(**dict(dict(k_cache=kc, v_cache=vc, heads=2, block_table=c["table"], page_size=16,
                                         moves=torch.zeros((1, 2, 3, 2), dtype=torch.int32, device=DEV), weights=w,
                                         positions=p), **kw))

    bad_move(ValueError, moves=torch.zeros((1, 2, 3, 2), device=DEV))
    bad_move(ValueError, moves=torch.zeros((2, 2, 3, 2), dtype=torch.int32, device=DEV))
    bad_move(ValueError, moves=torch.zeros((1, 2, 3, 3), dtype=torch.int32, device=DEV))
    bad_move(nv.NVFP4Error, moves=torch.zeros((1, 3, 3, 2), dtype=torch.int32, device=DEV))
    bad_move(ValueError, weights=w[:, :-1])
    bad_move(ValueError, positions=p.float())
    bad_move(nv.NVFP4Error, page_size=40)
