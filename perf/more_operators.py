"""Drafts in trees and a cache of bounded length, on the paged NVFP4 KV cache: what is timed, and its plain form.

Four operators, as a serving step runs them beside the append and the attention:

  tree     attention of a tree of drafted tokens over a sequence's cache: every draft sees the tokens
           before the tree and, of the tree, what its row of bits says (its ancestors and itself)
  weights  the attention weight that each cached token receives, per KV head, summed over the query
           rows and added to what it has received before (the log-sum-exps come from the attention)
  select   the tokens that a sequence keeps per KV head when it passes its budget: the first ones, the
           most recent ones and the heaviest; given as the moves that close the gaps
  move     moves of cached tokens within their sequence: the accepted path of a tree (one list for all
           heads) or the moves of select (a list per head), with the weights and positions

``run`` with ``own`` false computes them with elementary torch operations in 32 bits, with ``own`` true
through the library.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one user's chat, a small tree on a short context: the smallest call, latency counts
        dict(name="tree 1 x 16 on 700", kind="tree", seqs=1, qh=32, kvh=8, dim=128, page=16, m=16, m_hi=16, kv=700,
             kv_hi=700, window=0, empty=False, lens=1),
        # a busy server's batch: trees and contexts of very different sizes, one slot without a request
        dict(name="trees 32 x 26-63, ragged", kind="tree", seqs=32, qh=32, kvh=8, dim=128, page=16, m=26, m_hi=63,
             kv=300, kv_hi=16000, window=0, empty=True, lens=2),
        # sliding window layers, small heads
        dict(name="trees 24 x 20, window", kind="tree", seqs=24, qh=24, kvh=4, dim=64, page=32, m=20, m_hi=20,
             kv=3000, kv_hi=20000, window=4096, empty=False, lens=3),
        # a large tree on a long context, the KV cache heads of the benchmark (4 of 256)
        dict(name="tree 1 x 64 on 131072", kind="tree", seqs=1, qh=32, kvh=4, dim=256, page=64, m=64, m_hi=64,
             kv=131072, kv_hi=131072, window=0, empty=False, lens=4),
        # one token of one chat
        dict(name="weights 1 x 700", kind="weights", seqs=1, qh=32, kvh=8, dim=128, page=16, q=1, q_hi=1, kv=700,
             kv_hi=700, window=0, empty=False, lens=5),
        # a decode batch of chats of very different lengths, one finished slot among them
        dict(name="weights 64 ragged", kind="weights", seqs=64, qh=32, kvh=8, dim=128, page=16, q=1, q_hi=1, kv=64,
             kv_hi=16384, window=0, empty=True, lens=6),
        # a whole prompt before its first eviction
        dict(name="weights prompt 4096", kind="weights", seqs=1, qh=32, kvh=8, dim=128, page=64, q=4096, q_hi=4096,
             kv=0, kv_hi=0, window=0, empty=False, lens=7),
        # a decode batch at its budget: a page has filled up since the last time
        dict(name="select 64 x 2048 of 2049-2064", kind="select", seqs=64, kvh=8, page=16, kv=2049, kv_hi=2064,
             keep=2048, sinks=4, recent=256, stretch=3, lens=8),
        # prompts that were just read, of odd lengths: no positions yet but the places
        dict(name="select 16 x 4096, ragged", kind="select", seqs=16, kvh=8, page=16, kv=2000, kv_hi=16000, keep=4096,
             sinks=4, recent=512, stretch=0, lens=9),
        # one long prompt, the benchmark's KV heads
        dict(name="select 16384 of 131072", kind="select", seqs=1, kvh=4, page=64, kv=131072, kv_hi=131072, keep=16384,
             sinks=16, recent=1024, stretch=1, lens=10),
        # the accepted paths of a batch of trees: one list for all heads
        dict(name="move 32 paths of 6", kind="move", seqs=32, kvh=8, dim=128, page=16, kv=300, kv_hi=16000, keep=0,
             moves=6, heads=False, lens=11),
        # the long prompt's eviction: a list per head
        dict(name="move 14336 of 131072", kind="move", seqs=1, kvh=4, dim=256, page=64, kv=131072, kv_hi=131072,
             keep=16384, moves=14336, heads=True, lens=12),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "weights", "weights", "weights-rows", "select", "select", "move"])
    c = dict(kind=kind, page=rng.choice([16, 16, 32, 48, 64, 256]), lens=rng.randrange(1 << 30))
    kvh = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if kind in ("tree", "weights"):
        dim = rng.choice([64, 128, 256])
        qh = kvh * rng.choice([1, 2, 4, 5, 8])
        c.update(qh=qh, kvh=kvh, dim=dim, empty=rng.random() < 0.3)
        if kind == "tree":
            seqs = _log(rng, 1, 32)
            m = _log(rng, 2, 96)
            # (as many scores and cached values as the listed cases have)
            most = min(131072, 134217728 // (seqs * kvh * dim), (1 << 30) // (seqs * qh * m))
            hi = _log(rng, 32, max(64, most))
            return dict(c, seqs=seqs, m=max(1, m // 2), m_hi=m, kv=_log(rng, 1, hi), kv_hi=hi,
                        window=rng.choice([0, 0, 0, 24, 1024, 4096]))
        seqs = _log(rng, 1, 128)
        hi = _log(rng, 32, max(64, min(131072, 134217728 // (seqs * kvh * dim))))
        return dict(c, seqs=seqs, q=1, q_hi=rng.choice([1, 1, 1, 3, 8]), kv=_log(rng, 1, hi), kv_hi=hi,
                    window=rng.choice([0, 0, 0, _log(rng, 16, 8192)]))
    if kind == "weights-rows":  # prompts, and chunks on top of a context
        kvh = rng.choice([1, 2, 4, 8])
        qh = kvh * rng.choice([1, 4, 5, 8])
        seqs = _log(rng, 1, 8)
        q_hi = _log(rng, 24, max(32, min(4096, int(math.sqrt(4096 * 4096 * 32 / (seqs * qh))))))
        before = max(0, 4096 * 4096 * 32 // (seqs * qh * q_hi) - q_hi)
        kv_hi = rng.choice([0, _log(rng, 64, max(65, min(32768, before)))])
        return dict(c, kind="weights", seqs=seqs, qh=qh, kvh=kvh, dim=rng.choice([64, 128, 256]), empty=False,
                    q=_log(rng, 9, q_hi), q_hi=q_hi, kv=min(kv_hi, 33), kv_hi=kv_hi, window=rng.choice([0, 0, 512]))
    if kind == "select":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 40, max(64, min(131072, (1 << 20) // (seqs * kvh))))
        keep = max(24, _log(rng, 24, hi))
        sinks = rng.choice([0, 1, 4, 16])
        return dict(c, seqs=seqs, kvh=kvh, kv=max(1, hi - rng.choice([7, hi // 2, hi - 1])), kv_hi=hi, keep=keep,
                    sinks=sinks, recent=_log(rng, 1, keep - sinks), stretch=rng.choice([0, 1, 1, 4]))
    dim = rng.choice([64, 128, 256])
    if rng.random() < 0.5:
        return dict(c, seqs=_log(rng, 1, 64), kvh=kvh, dim=dim, kv=100, kv_hi=_log(rng, 200, 4000), keep=0,
                    moves=_log(rng, 1, 20), heads=False)
    seqs = _log(rng, 1, 16)
    hi = _log(rng, 600, max(800, min(131072, 134217728 // (seqs * kvh * dim))))
    keep = _log(rng, 64, hi // 2)
    return dict(c, seqs=seqs, kvh=kvh, dim=dim, kv=max(keep + 20, hi // 2), kv_hi=max(keep + 20, hi), keep=keep,
                moves=_log(rng, 1, min(keep, 14336)), heads=True)


def _lengths(case):
    """Query tokens and cached tokens (the query's own among them) of each sequence."""
    r = random.Random(case["lens"])
    lo, hi = (case["m"], case["m_hi"]) if case["kind"] == "tree" else (case.get("q", 0), case.get("q_hi", 0))
    q, kv = [], []
    for _ in range(case["seqs"]):
        nq = _log(r, lo, hi) if hi else 0
        before = _log(r, max(1, case["kv"]), case["kv_hi"]) if case["kv_hi"] else 0
        # one decoded token: kv counts it; several, or a tree: they come on top of the context
        q.append(nq)
        kv.append(before if case["kind"] != "tree" and hi <= 1 else before + nq)
    if case.get("empty") and case["seqs"] > 1:
        kv[case["seqs"] // 2] = 0  # a slot without a request: its rows have no key
    return q, kv


def _trees(case, q_lens):
    """The ancestors of every draft, itself among them: for each sequence a truth table [m, m]."""
    r = random.Random(case["lens"] + 1)
    tables = []
    for m in q_lens:
        t = np.zeros((m, m), dtype=bool)
        for i in range(m):
            # several first tokens, then each a continuation of some earlier one, of a late one more often
            parent = -1 if i < 2 or r.random() < 0.1 else int(i * math.sqrt(r.random()))
            if parent >= 0:
                t[i] = t[parent]
            t[i, i] = True
        tables.append(t)
    return tables


# ------------------------------------------------------------ the inputs ---

def _codes(a):
    """Nearest E2M1 code of magnitudes a, ties to the even code."""
    c = (a > 0.25).to(torch.uint8)
    for i, edge in enumerate((0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        c += (a >= edge) if i % 2 == 0 else (a > edge)
    return c


def _cache(g, rows, dim):
    """An NVFP4 cache tensor of `rows` rows: channels of unequal size, as keys and values have."""
    packed = torch.empty((1, rows, dim // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((1, rows, dim // 16), dtype=torch.uint8, device=DEV)
    channel = torch.exp(0.5 * torch.randn(dim, generator=g, device=DEV))
    G = (7.0 * channel.max() / 2688.0).reshape(1)
    for a in range(0, rows, 1 << 19):
        b = min(rows, a + (1 << 19))
        x = (torch.randn((b - a, dim), generator=g, device=DEV) * channel).unflatten(1, (-1, 16))
        s = (x.abs().amax(-1) / (6.0 * G)).clamp(max=448.0).to(torch.float8_e4m3fn)
        f = s.float()
        y = x * torch.where(f > 0, 1.0 / (f * G), torch.zeros_like(f))[..., None]
        code = (_codes(y.abs()) + 8 * torch.signbit(y).to(torch.uint8)).flatten(1)
        packed[0, a:b] = code[:, ::2] | (code[:, 1::2] << 4)
        scales[0, a:b] = s.view(torch.uint8)
    return packed, scales, G


def _decode(packed, scales, G):
    """fp32 values of NVFP4 bytes: packed [..., D/2], scales [..., D/16]."""
    pair = torch.tensor([(E2M1[b & 15], E2M1[b >> 4]) for b in range(256)], device=packed.device)
    v = pair[packed.int()].flatten(-2).unflatten(-1, (-1, 16))
    return ((v * scales.view(torch.float8_e4m3fn).float()[..., None]) * G).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    kvh, page, seqs = case["kvh"], case["page"], case["seqs"]
    q_lens, kv_lens = _lengths(case)
    pages = [-(-m // page) for m in kv_lens]
    pool = sum(pages) + 5
    order = torch.randperm(pool, generator=g, device=DEV).int()
    table = torch.full((seqs, max(1, max(pages))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = order[at:at + m]
        at += m
    s["table"] = table
    s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    tokens = s["tokens"] = pool * page
    kind = case["kind"]
    if kind in ("tree", "weights"):
        qh, dim, n = case["qh"], case["dim"], sum(q_lens)
        s["q"] = (1.5 * torch.randn((n, qh, dim), generator=g, device=DEV)).bfloat16()
        cu = torch.zeros(seqs + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(q_lens, dtype=torch.int32).cumsum(0)
        s["cu_q"], s["max_q"] = cu.to(DEV), max(q_lens)
        s["k_cache"] = _cache(g, tokens * kvh, dim)
    if kind == "tree":
        s["v_cache"] = _cache(g, tokens * kvh, dim)
        words = -(-max(q_lens) // 32)
        bits = np.zeros((n, 32 * words), dtype=bool)
        for first, t in zip(cu.tolist(), _trees(case, q_lens)):
            bits[first:first + len(t), :len(t)] = t
        s["mask"] = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)
    elif kind == "weights":
        # what the tokens have received so far, and the log-sum-exps that the attention left
        s["weights"] = torch.exp(2.0 * torch.randn((kvh, tokens), generator=g, device=DEV))
        s["out"] = torch.zeros((kvh, tokens), device=DEV)
        s["lse"] = _lse(s)
    elif kind == "select":
        # heavy tails, and tokens that never received any
        w = torch.exp(2.0 * torch.randn((kvh, tokens), generator=g, device=DEV))
        s["weights"] = torch.where(torch.rand((kvh, tokens), generator=g, device=DEV) < 0.1, 0.0, w)
        s["positions"] = s["next"] = None
        if case["stretch"]:
            # the positions of what earlier evictions left, in the order that the moves left them in
            s["positions"] = torch.zeros((kvh, tokens), dtype=torch.int32, device=DEV)
            s["next"] = s["kv_lens"] * case["stretch"]
            for b, m in enumerate(kv_lens):
                spread = (torch.arange(m, device=DEV) * case["stretch"]).int()
                newest = min(m, case["recent"])
                spread[m - newest:] = m * case["stretch"] - newest + torch.arange(newest, device=DEV, dtype=torch.int32)
                mixed = torch.rand((kvh, m), generator=g, device=DEV).argsort(1)
                s["positions"][:, _slots(s, b, m)] = spread[mixed]
        s["cap"] = max(1, min(case["keep"], table.shape[1] * page - case["keep"]))
    else:
        dim = case["dim"]
        s["k_cache"], s["v_cache"] = _cache(g, tokens * kvh, dim), _cache(g, tokens * kvh, dim)
        s["weights"] = torch.exp(2.0 * torch.randn((kvh, tokens), generator=g, device=DEV))
        s["positions"] = torch.randint(0, 1 << 20, (kvh, tokens), generator=g, device=DEV, dtype=torch.int32)
        s["moves"] = _moves(case, kv_lens, g)
        s["to"] = _rows_of(s)[0]
        s["ids"] = s["to"].int()
    return s


def _moves(case, kv_lens, g):
    """(source, destination) places, int32 [seqs, lists, moves, 2], -1 behind the last of a list."""
    lists = case["kvh"] if case["heads"] else 1
    moves = torch.full((case["seqs"], lists, case["moves"], 2), -1, dtype=torch.int32, device=DEV)
    for b, m in enumerate(kv_lens):
        if case["heads"]:
            # gaps among the kept places, and the tokens behind them that stay, both in order
            k = min(case["moves"], case["keep"], m - case["keep"])
            src = torch.rand((lists, m - case["keep"]), generator=g, device=DEV).argsort(1)[:, :k].sort(1)[0]
            dst = torch.rand((lists, case["keep"]), generator=g, device=DEV).argsort(1)[:, :k].sort(1)[0]
            src = src + case["keep"]
        else:
            # a path through a tree listed level by level: its tokens lie behind the places they go to
            k = case["moves"]
            wide = min(64, m - k)
            src = torch.rand((1, wide - k), generator=g, device=DEV).argsort(1)[:, :k].sort(1)[0] + m - wide + k
            dst = (m - wide + torch.arange(k, device=DEV))[None]
        moves[b, :, :k, 0], moves[b, :, :k, 1] = src.int(), dst.int()
    return moves


# ------------------------------------------------------------ plain forms --

def _slots(s, b, m):
    """Cache tokens of the first m tokens of sequence b."""
    t = torch.arange(m, device=DEV)
    return s["table"][b].long()[t // s["page"]] * s["page"] + t % s["page"]


def _all_slots(s):
    """Cache tokens [seqs, places] of every place of the table (anything past a sequence's end)."""
    return (s["table"].clamp(min=0).long()[:, :, None] * s["page"] + torch.arange(s["page"], device=DEV)).flatten(1)


def _queries(s):
    """The queries of each sequence, padded to the longest: (index [seqs, max_q], their number [seqs])."""
    first, count = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    at = first[:, None] + torch.arange(s["max_q"], device=DEV)
    return at.clamp(max=s["q"].shape[0] - 1), count


def _scores(s, slots, at, seen):
    """fp32 scores [seqs, kvh, group, rows, places] of the queries `at`, -inf where not seen [seqs, rows, places]."""
    qh, kvh, dim = s["qh"], s["kvh"], s["dim"]
    packed, scales, G = s["k_cache"]
    k = _decode(packed.view(-1, kvh, dim // 2)[slots], scales.view(-1, kvh, dim // 16)[slots], G)
    k = k.transpose(1, 2).contiguous()  # [seqs, kvh, places, dim]
    q = s["q"].float()[at].unflatten(2, (kvh, qh // kvh)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (qh // kvh, at.shape[1])) * (dim ** -0.5)
    return x.masked_fill_(~seen[:, None, None], -math.inf)


def _seen(s, places, at, count, rows):
    """Which places the query rows [r0, r1) see: causal, within the window."""
    i = torch.arange(*rows, device=DEV)
    place = s["kv_lens"].long()[:, None] - count[:, None] + i  # each query's own
    t = torch.arange(places, device=DEV)
    seen = (t <= place[..., None]) & (t < s["kv_lens"][:, None, None])
    if s["window"]:
        seen &= t > place[..., None] - s["window"]
    return seen & (i < count[:, None])[..., None]


def _pieces(s, places):
    """Runs of query rows whose scores take up to about 2 GiB."""
    step = max(1, (1 << 29) // (s["table"].shape[0] * s["qh"] * places))
    return [(a, min(s["max_q"], a + step)) for a in range(0, s["max_q"], step)]


def _lse(s):
    slots = _all_slots(s)
    at, count = _queries(s)
    n = s["q"].shape[0]
    lse = torch.full((n + 1, s["qh"]), -math.inf, device=DEV)
    for a, b in _pieces(s, slots.shape[1]):
        x = _scores(s, slots, at[:, a:b], _seen(s, slots.shape[1], at, count, (a, b)))
        z = torch.logsumexp(x, -1).permute(0, 3, 1, 2).flatten(2)
        real = torch.arange(a, b, device=DEV) < count[:, None]
        lse[torch.where(real, at[:, a:b], n)] = z
    return lse[:n].contiguous()


def _plain_weights(s):
    slots = _all_slots(s)
    places = slots.shape[1]
    at, count = _queries(s)
    total = torch.zeros((slots.shape[0], s["kvh"], places), device=DEV)
    for a, b in _pieces(s, places):
        x = _scores(s, slots, at[:, a:b], _seen(s, places, at, count, (a, b)))
        z = s["lse"][at[:, a:b]].unflatten(2, (s["kvh"], -1)).permute(0, 2, 3, 1)[..., None]
        total += torch.exp(x - torch.where(z == -math.inf, 0.0, z)).sum((2, 3))
    t = torch.arange(places, device=DEV)
    before = s["weights"][:, slots].transpose(0, 1)
    fresh = t >= s["kv_lens"][:, None] - count[:, None]  # the queries' own tokens have received nothing yet
    total += torch.where(fresh[:, None], 0.0, before)
    b, t = (t < s["kv_lens"][:, None]).nonzero(as_tuple=True)
    s["out"][:, slots[b, t]] = total[b, :, t].T
    return {"weights": s["out"]}


def _plain_tree(s):
    qh, kvh, dim, seqs, mq = s["qh"], s["kvh"], s["dim"], s["seqs"], s["max_q"]
    slots = _all_slots(s)
    t = torch.arange(slots.shape[1], device=DEV)
    at, count = _queries(s)
    j = torch.arange(32 * s["mask"].shape[1], device=DEV)
    bits = ((s["mask"][:, j // 32] >> (j % 32)) & 1).bool()[at]  # [seqs, rows, drafts]
    base = s["kv_lens"].long() - count  # the first draft's place
    bits &= (j < count[:, None])[:, None] & (base[:, None] + j >= 0)[:, None]
    if s["window"]:
        # of the tokens before the tree and the row's drafts, in this order, the last ones
        behind = bits.flip(2).cumsum(2).flip(2)
        in_row = behind[..., 0]
        bits &= behind <= s["window"]
        start = base[:, None] - (s["window"] - in_row).clamp(min=0)
    else:
        start = torch.zeros_like(at)
    seen = (t >= start[..., None]) & (t < base[:, None, None])
    draft = t - base[:, None]
    inside = (draft >= 0) & (draft < count[:, None])
    pick = draft.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, mq, -1)
    seen |= inside[:, None] & bits.gather(2, pick)
    seen &= t < s["kv_lens"][:, None, None]
    x = _scores(s, slots, at, seen)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    del x
    total = p.sum(-1, keepdim=True)
    packed, scales, G = s["v_cache"]
    v = _decode(packed.view(-1, kvh, dim // 2)[slots], scales.view(-1, kvh, dim // 16)[slots], G)
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2).contiguous()).unflatten(2, (qh // kvh, mq))
    o = o / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]
    n = s["q"].shape[0]
    b = torch.repeat_interleave(torch.arange(seqs, device=DEV), count, output_size=n)
    i = torch.arange(n, device=DEV) - s["cu_q"][:-1].long()[b]
    return {"out": o.permute(0, 3, 1, 2, 4)[b, i].flatten(1, 2).bfloat16(),
            "lse": lse.permute(0, 3, 1, 2)[b, i].flatten(1, 2)}


def _plain_select(s):
    keep, cap = s["keep"], s["cap"]
    slots = _all_slots(s)
    t = torch.arange(slots.shape[1], device=DEV)
    lens = s["kv_lens"][:, None, None]
    w = s["weights"][:, slots].transpose(0, 1)  # [seqs, kvh, places]
    pos = t.expand_as(w) if s["positions"] is None else s["positions"][:, slots].transpose(0, 1)
    after = lens if s["positions"] is None else s["next"][:, None, None]
    key = torch.where(torch.isnan(w), -math.inf, w).double().clamp(-1e300, 1e300)
    key = torch.where((pos < s["sinks"]) | (pos >= after - s["recent"]), math.inf, key)
    key = torch.where(t < lens, key, -math.inf)
    order = torch.sort(key, dim=2, descending=True, stable=True)[1]
    kept = torch.zeros_like(order, dtype=torch.bool).scatter_(2, order[..., :keep], True) & (t < lens)
    gap, mover = (t < keep) & (t < lens) & ~kept, (t >= keep) & kept
    moves = torch.full(order.shape[:2] + (cap + 1, 2), -1, dtype=torch.int32, device=DEV)
    place = t.int().expand_as(order)
    for j, which in ((0, mover), (1, gap)):
        rank = torch.where(which, which.cumsum(2) - 1, cap)
        moves[..., j].scatter_(2, rank, torch.where(which, place, -1))
    return {"moves": moves[:, :, :cap].contiguous(), "lens": s["kv_lens"].clamp(max=keep)}


def _rows_of(s):
    """Cache rows (token, head) that the moves go to and come from: flat, in the order of the lists."""
    kvh = s["kvh"]
    moves = s["moves"].long().expand(-1, kvh, -1, -1)  # [seqs, kvh, moves, 2]
    slot = _all_slots(s)[torch.arange(moves.shape[0], device=DEV)[:, None, None, None], moves.clamp(min=0)]
    row = slot * kvh + torch.arange(kvh, device=DEV)[None, :, None, None]
    real = moves[..., 0] >= 0
    return row[..., 1][real], row[..., 0][real]


def _plain_move(s):
    to, come = _rows_of(s)
    for packed, scales, _ in (s["k_cache"], s["v_cache"]):
        packed[0, to] = packed[0, come]
        scales[0, to] = scales[0, come]
    for x in (s["weights"], s["positions"]):
        x[to % s["kvh"], to // s["kvh"]] = x[come % s["kvh"], come // s["kvh"]]
    out = {"weights": s["weights"], "positions": s["positions"]}
    for name in ("k", "v"):
        packed, scales, G = s[name + "_cache"]
        out[name] = _decode(packed[0, s["to"]], scales[0, s["to"]], G).bfloat16()
    return out


def run(state):
    s = state
    if not own:
        return {"tree": _plain_tree, "weights": _plain_weights, "select": _plain_select, "move": _plain_move}[s["kind"]](s)
    import precision_moe_gemm_amd as nv
    kvh, page = s["kvh"], s["page"]
    if s["kind"] == "select":
        moves, lens = nv.nvfp4_kv_select(s["weights"], s["table"], s["kv_lens"], page, s["keep"], positions=s["positions"],
                                         next_positions=s["next"], sinks=s["sinks"], recent=s["recent"], cap=s["cap"])
        return {"moves": moves, "lens": lens}
    kc = nv.NVFP4Tensor(*s["k_cache"], s["tokens"] * kvh, s["dim"])
    if s["kind"] == "weights":
        out = nv.nvfp4_kv_weights(s["q"], s["lse"], kc, kvh, s["table"], s["kv_lens"], page, s["out"], weights=s["weights"],
                                  cu_q=s["cu_q"] if s["max_q"] > 1 else None, max_q=s["max_q"], window=s["window"])
        return {"weights": out}
    vc = nv.NVFP4Tensor(*s["v_cache"], s["tokens"] * kvh, s["dim"])
    if s["kind"] == "tree":
        out, lse = nv.nvfp4_kv_attention_tree(s["q"], kc, vc, kvh, s["table"], s["kv_lens"], page, s["cu_q"], s["mask"],
                                              max_q=s["max_q"], window=s["window"], return_lse=True)
        return {"out": out, "lse": lse}
    nv.nvfp4_kv_move(kc, vc, kvh, s["table"], page, s["moves"], weights=s["weights"], positions=s["positions"])
    return {"weights": s["weights"], "positions": s["positions"], "k": nv.nvfp4_gather_dequantize(kc, s["ids"]),
            "v": nv.nvfp4_gather_dequantize(vc, s["ids"])}


def work(case):
    kvh = case["kvh"]
    q_lens, kv_lens = _lengths(case)
    if case["kind"] == "select":
        per = 4 + (4 if case["stretch"] else 0)
        chosen = sum(min(case["keep"], m - case["keep"]) for m in kv_lens if m > case["keep"])
        return {"bytes": sum(kv_lens) * kvh * per + 8 * chosen * kvh, "flops": 4 * sum(kv_lens) * kvh}
    dim = case["dim"]
    row = dim // 2 + dim // 16  # one NVFP4 row
    if case["kind"] == "move":
        lists = kvh if case["heads"] else 1
        count = [min(case["moves"], case["keep"], m - case["keep"]) if case["heads"] else case["moves"] for m in kv_lens]
        # each list, and for each move the rows and two numbers read and written; then the rows read back in bf16
        return {"bytes": sum(count) * (8 * lists + kvh * (2 * (2 * row + 8) + 2 * (row + 2 * dim))), "flops": 0}
    qh, n = case["qh"], sum(q_lens)
    if case["kind"] == "tree":
        pairs = tokens = 0
        for nq, m, t in zip(q_lens, kv_lens, _trees(case, q_lens)):
            base = m - nq
            if base < 0:
                continue  # (an empty slot)
            drafts = t.sum(1)
            w = case["window"] or 1 << 40
            before = np.minimum(base, np.maximum(0, w - drafts))
            pairs += int((before + np.minimum(drafts, w)).sum())
            tokens += int(before.max()) + nq
        words = -(-max(q_lens) // 32)
        return {"bytes": n * (qh * (4 * dim + 4) + 4 * words) + tokens * kvh * 2 * row, "flops": 4 * pairs * qh * dim}
    pairs = tokens = 0
    for nq, m in zip(q_lens, kv_lens):
        ends = [min(m, max(0, m - nq + i + 1)) for i in range(nq)]
        lo = [max(0, m - nq + i + 1 - case["window"]) if case["window"] else 0 for i in range(nq)]
        pairs += sum(max(0, e - a) for a, e in zip(lo, ends))
        tokens += max(0, max(ends) - min(lo))
    return {"bytes": n * qh * (2 * dim + 4) + tokens * kvh * row + sum(kv_lens) * kvh * 8,
            "flops": 2 * pairs * qh * dim}


# ------------------------------------------------------------ 64 bits ------

def _exact_rows(s, name, slot):
    """float64 values [tokens, kvh, D] of a cache."""
    packed, scales, G = s[name]
    kvh, dim = s["kvh"], s["dim"]
    value = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    p = packed.view(-1, kvh, dim // 2)[slot]
    x = torch.empty(p.shape[:2] + (dim,), dtype=torch.float64, device=DEV)
    x[..., ::2], x[..., 1::2] = value[(p & 15).long()], value[(p >> 4).long()]
    sc = scales.view(-1, kvh, dim // 16)[slot].view(torch.float8_e4m3fn).to(torch.float64)
    return x * sc.repeat_interleave(16, 2) * float(G)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    kvh, page = case["kvh"], case["page"]
    q_lens, kv_lens = _lengths(case)
    if case["kind"] == "select":
        return None  # (whole numbers, which the plain form gives exactly)
    if case["kind"] == "move":
        w, pos, out = s["weights"].cpu().numpy(), s["positions"].cpu().numpy(), {"k": [], "v": []}
        old_w, old_pos = w.copy(), pos.copy()
        moves, table = s["moves"].cpu().numpy(), s["table"].cpu().numpy()
        if moves.size > 1 << 18:
            return None
        come = []
        for b in range(case["seqs"]):
            for h in range(kvh):
                for src, dst in moves[b, h if case["heads"] else 0]:
                    if src >= 0:
                        x, y = (int(table[b, t // page]) * page + int(t % page) for t in (src, dst))
                        w[h, y], pos[h, y] = old_w[h, x], old_pos[h, x]
                        come.append((x, h))
        come = torch.tensor(come, device=DEV)
        for name in ("k", "v"):
            out[name] = torch.cat([_exact_rows(s, name + "_cache", c[:, 0])[torch.arange(len(c), device=DEV), c[:, 1]]
                                   for c in come.split(1 << 14)])
        return {"weights": torch.from_numpy(w).to(f64), "positions": torch.from_numpy(pos), **out}
    qh = case["qh"]
    group = qh // kvh
    if max(a * b for a, b in zip(q_lens, kv_lens)) * qh > 1 << 31:
        return None
    trees = _trees(case, q_lens) if case["kind"] == "tree" else None
    out, lse, at = [], [], 0
    weights = s["out"].to(f64) if case["kind"] == "weights" else None
    for b, (nq, m) in enumerate(zip(q_lens, kv_lens)):
        q = s["q"][at:at + nq].to(f64)
        z_given = s["lse"][at:at + nq].to(f64) if case["kind"] == "weights" else None
        at += nq
        slot = _slots(s, b, m)
        K = _exact_rows(s, "k_cache", slot)
        if case["kind"] == "tree":
            hide = torch.ones((nq, m), dtype=torch.bool, device=DEV)
            base = m - nq
            for i in range(nq if m else 0):
                row = list(range(base)) + [base + j for j in range(nq) if trees[b][i, j]]
                hide[i, torch.tensor(row[-case["window"]:] if case["window"] else row, device=DEV)] = False
            V = _exact_rows(s, "v_cache", slot)
            o = torch.zeros((nq, qh, case["dim"]), dtype=f64, device=DEV)
            z = torch.full((nq, qh), -math.inf, dtype=f64, device=DEV)
        else:
            t, place = torch.arange(m, device=DEV), torch.arange(nq, device=DEV) + (m - nq)
            hide = t[None] > place[:, None]
            if case["window"]:
                hide = hide | (t[None] <= place[:, None] - case["window"])
            got = s["weights"].to(f64)[:, slot]
            got[:, max(0, m - nq):] = 0.0
        for h in range(qh if m else 0):
            for r in range(0, nq, 1024):
                x = (q[r:r + 1024, h] @ K[:, h // group].T) / math.sqrt(case["dim"])
                x[hide[r:r + 1024]] = -math.inf
                if case["kind"] == "tree":
                    z[r:r + 1024, h] = torch.logsumexp(x, 1)
                    o[r:r + 1024, h] = torch.softmax(x, 1) @ V[:, h // group]
                else:
                    zz = z_given[r:r + 1024, h, None]
                    got[h // group] += torch.exp(x - torch.where(zz > -math.inf, zz, 0.0)).sum(0)
        if case["kind"] == "tree":
            out.append(o)
            lse.append(z)
        else:
            weights[:, slot] = got
    if case["kind"] == "tree":
        return {"out": torch.cat(out), "lse": torch.cat(lse)}
    return {"weights": weights}
