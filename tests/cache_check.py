"""Plain 64-bit forms of the operators for trees of drafts and for caches of bounded length, for the parity
tests, and the error bounds that their kernels are held to."""
import numpy as np
import torch

from tests.attn_check import STEP, values


def bits_of(mask):
    """Truth table [n, 32 words] of int32 mask rows."""
    m = mask.cpu().contiguous().numpy().view(np.uint32)
    return ((m[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).astype(bool).reshape(len(m), 32 * m.shape[1])


def mask_of(bits):
    """int32 mask rows of a truth table (padded to whole words)."""
    bits = np.asarray(bits, dtype=bool)
    pad = -bits.shape[1] % 32
    bits = np.pad(bits, ((0, 0), (0, pad)))
    return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).reshape(len(bits), -1).copy())


def tree_seen(bits, m, kv, window):
    """Places that each of a sequence's m drafts sees; bits: their rows of the truth table."""
    base = kv - m
    seen = []
    for i in range(m):
        t = list(range(max(0, base))) + [base + j for j in range(min(m, bits.shape[1])) if bits[i, j] and base + j >= 0]
        seen.append(t[-window:] if window else t)
    return seen


def causal_seen(m, kv, causal, window):
    """Places that each of a sequence's m query rows sees."""
    seen = []
    for i in range(m):
        e = min(kv, max(0, kv - m + i + 1)) if causal else kv
        seen.append(list(range(max(0, kv - m + i + 1 - window) if window else 0, e)))
    return seen


def _cache_values(cache, heads, page):
    pool = cache.rows // heads // page
    return values(cache.packed[0], cache.scales[0]).view(pool, page, heads, -1) * float(cache.global_[0]), pool


def _offsets(kv_lens, cu_q):
    return list(range(len(kv_lens) + 1)) if cu_q is None else cu_q.cpu().tolist()


def attention_over(seen, q, k_cache, v_cache, heads, table, page, first, scale=None):
    """(out, lse, out_tol, lse_tol) in float64 on the CPU, rows of one sequence whose row i sees places seen[i];
    the bounds are those of attn_check.attention."""
    n, qh, D = len(seen), q.shape[1], q.shape[2]
    g = qh // heads
    scale = D ** -0.5 if scale is None else scale
    qd = q.cpu().double()
    K, pool = _cache_values(k_cache, heads, page)
    V, _ = _cache_values(v_cache, heads, page)
    out, tol = torch.zeros((n, qh, D), dtype=torch.float64), torch.zeros((n, qh, D), dtype=torch.float64)
    lse, ltol = torch.full((n, qh), -np.inf, dtype=torch.float64), torch.zeros((n, qh), dtype=torch.float64)
    for i, t in enumerate(seen):
        t = torch.tensor(t, dtype=torch.long)
        if len(t):
            pg = table.cpu()[t // page].long()
            ok = (pg >= 0) & (pg < pool)
            t, pg = t[ok], pg[ok]
        if not len(t):
            continue
        for h in range(heads):
            rows = slice(h * g, (h + 1) * g)
            kk, vv = K[pg, t % page, h], V[pg, t % page, h]
            x = qd[first + i, rows]
            sc = (x @ kk.T) * scale
            S = ((x.abs() @ kk.abs().T) * scale).amax(1)
            S2 = D * x.abs().amax(1) * kk.abs().max() * scale
            z = torch.logsumexp(sc, 1)
            p = torch.exp(sc - z[:, None])
            o = p @ vv
            out[i, rows], lse[i, rows] = o, z
            rel = (D + 4) * STEP * S + STEP * S2
            run = 2 * (len(t) / 8 + 64) * STEP
            tol[i, rows] = (o.abs() * 2.0 ** -8 + (p @ vv.abs()) * (2.0 ** -11 + 2 * rel + run)[:, None]
                            + 2.0 ** -31 * vv.abs().sum(0) * p.amax(1)[:, None])
            ltol[i, rows] = rel + run + 4 * STEP * (z.abs() + sc.abs().amax(1))
    return out, lse, tol, ltol


def tree_attention(q, k_cache, v_cache, heads, table, kv_lens, page, cu_q, mask, scale=None, window=0):
    """(out, lse, out_tol, lse_tol) of nvfp4_kv_attention_tree."""
    bits, cu = bits_of(mask), _offsets(kv_lens, cu_q)
    parts = []
    for b, kv in enumerate(kv_lens.cpu().tolist()):
        m = cu[b + 1] - cu[b]
        seen = tree_seen(bits[cu[b]:cu[b + 1]], m, kv, window)
        parts.append(attention_over(seen, q, k_cache, v_cache, heads, table[b], page, cu[b], scale))
    return tuple(torch.cat(x) for x in zip(*parts))


def received(q, lse, k_cache, heads, table, kv_lens, page, before, cu_q=None, scale=None, causal=True, window=0):
    """(weights, tol, written) of nvfp4_kv_weights: float64 [heads, tokens] on the CPU, NaN where no token of a
    sequence lies; `written`: where one does.

    Bounds.  A score is off, relatively in its exponential, by what attn_check.attention derives: (D + 4) steps of
    S = sum |q k| scale, and a step of S2 = D max |q| max |k| scale for elements of q far below their row's largest.
    Its factor, the log-sum-exp in units of ln 2 and the fused multiply-add round once each: 3 steps of
    |s| + |lse|, doubled for the constant 1 / ln 2.  The exponential is off by one unit in the last place (two
    steps).  The weights of R rows are added in fp32 with at most R additions of partial sums no larger than the
    whole, and once more to what was there: R + 4 steps of the sum and 2 of the result."""
    n, qh, D = q.shape
    g = qh // heads
    scale = D ** -0.5 if scale is None else scale
    qd, z = q.cpu().double(), lse.cpu().double()
    K, pool = _cache_values(k_cache, heads, page)
    tokens = pool * page
    out, tol = torch.full((heads, tokens), np.nan, dtype=torch.float64), torch.zeros((heads, tokens), dtype=torch.float64)
    cu = _offsets(kv_lens, cu_q)
    for b, kv in enumerate(kv_lens.cpu().tolist()):
        m = cu[b + 1] - cu[b]
        t = torch.arange(kv)
        pg = table.cpu()[b][t // page].long() if kv else t
        ok = (pg >= 0) & (pg < pool)
        t, pg = t[ok], pg[ok]
        slot = pg * page + t % page
        fresh = t >= kv - m
        see = torch.zeros((m, kv), dtype=torch.bool)
        for i, places in enumerate(causal_seen(m, kv, causal, window)):
            see[i, places] = True
        see = see[:, t]
        for h in range(heads):
            w = torch.zeros(len(t), dtype=torch.float64) if before is None else before.cpu().double()[h, slot]
            w = torch.where(fresh, 0.0, w)
            kk = K[pg, t % page, h]
            x = qd[cu[b]:cu[b + 1], h * g:(h + 1) * g].reshape(m * g, D)
            zz = z[cu[b]:cu[b + 1], h * g:(h + 1) * g].reshape(m * g, 1)
            use = torch.isfinite(zz) & see.repeat_interleave(g, 0) & torch.isfinite(x).all(1, keepdim=True)
            x, zz = torch.nan_to_num(x, 0.0, 0.0, 0.0), torch.where(torch.isfinite(zz), zz, 0.0)
            sc = (x @ kk.T) * scale
            p = torch.where(use, torch.exp(sc - zz), 0.0)
            S = (x.abs() @ kk.abs().T) * scale
            S2 = D * x.abs().amax(1, keepdim=True) * (kk.abs().max() if len(t) else 0.0) * scale if m else S
            rel = (D + 4) * STEP * S + STEP * S2 + 6 * STEP * (sc.abs() + zz.abs()) + 2 * STEP
            total = p.sum(0)
            out[h, slot] = w + total
            tol[h, slot] = (p * 1.01 * rel).sum(0) + (m * g + 4) * STEP * total + 2 * STEP * (w.abs() + total) + 2.0 ** -120
    return out, tol, ~torch.isnan(out)


def chosen(weights, positions, table, kv_lens, page, keep, next_positions, sinks, recent, cap, pool=None):
    """(moves, lens) of nvfp4_kv_select, numpy."""
    w, table = weights.cpu().double().numpy(), table.cpu().numpy()
    pos = None if positions is None else positions.cpu().numpy()
    heads = w.shape[0]
    pool = w.shape[1] // page if pool is None else pool
    lens = kv_lens.cpu().tolist()
    moves = np.full((len(lens), heads, cap, 2), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        if n <= keep:
            continue
        t = np.arange(n)
        pg = table[b][t // page]
        ok = (pg >= 0) & (pg < pool)
        slot = np.where(ok, pg, 0) * page + t % page
        for h in range(heads):
            x = w[h, slot].copy()
            x[np.isnan(x)] = -np.inf
            p = t if pos is None else pos[h, slot].astype(np.int64)
            end = n if pos is None else int(next_positions[b])
            first = (p < sinks) | (p >= end - recent)
            # classes: kept anyway, by weight, in no page; of equals the lowest place (lexsort: last key first)
            cls = np.where(ok, np.where(first, 0, 1), 2)
            x[cls != 1] = 0
            order = np.lexsort((t, -x, cls))
            kept = np.zeros(n, dtype=bool)
            kept[order[:keep]] = True
            src, dst = t[keep:][kept[keep:]], t[:keep][~kept[:keep]]
            moves[b, h, :len(src), 0], moves[b, h, :len(dst), 1] = src, dst
    return moves, np.minimum(lens, keep)


def moved(arrays, moves, table, page, heads, pool=None):
    """Numpy copies of arrays indexed [token, head, ...] after the moves, every source read first."""
    moves, table = np.asarray(moves), np.asarray(table)
    out = [a.copy() for a in arrays]
    tokens = arrays[0].shape[0]
    pool = tokens // page if pool is None else pool
    for b in range(moves.shape[0]):
        for h in range(heads):
            for src, dst in moves[b, h if moves.shape[1] > 1 else 0].tolist():
                if src < 0 or src >= table.shape[1] * page or not 0 <= dst < table.shape[1] * page:
                    continue
                p, q = int(table[b, src // page]), int(table[b, dst // page])
                if not (0 <= p < pool and 0 <= q < pool):
                    continue
                for a, o in zip(arrays, out):
                    o[q * page + dst % page, h] = a[p * page + src % page, h]
    return out
