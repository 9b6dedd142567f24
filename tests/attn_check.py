"""Plain 64-bit forms of the attention-side operators, for the parity tests, and the error bounds
that their kernels are held to."""
import numpy as np
import torch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
STEP = 2.0 ** -24  # half a step of fp32, relative


def values(packed, scales):
    """float64 code * scale of NVFP4 rows on the CPU (without the global): packed [..., D/2]."""
    packed = packed.cpu()
    v = torch.stack([E2M1[(packed & 15).long()], E2M1[(packed >> 4).long()]], -1).flatten(-2)
    s = scales.cpu().view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(16, -1)


def attention(q, k_cache, v_cache, heads, table, kv_lens, page, cu_q=None, scale=None, causal=True, window=0):
    """(out, lse, out_tol, lse_tol), float64 on the CPU, of nvfp4_kv_attention's formula.  A page that is
    not one of the cache is skipped.

    Bounds.  A score is a sum of D exact products in fp32 (the matrix instruction may round every one
    of them, in any order) and two more roundings: off by at most (D + 4) steps of sum |q k| scale = S;
    q's elements below 2^-16 of their row's largest are off by 2^-25 of that largest: one more step of
    D max |q| max |k| scale, taken as S2.  exp of it is off by that, relatively, in numerator and
    denominator both.  p is rounded to f16 (2^-11: a value in [1, 2) is a multiple of 2^-10 there, so
    off by at most 2^-11, and by as much relatively at 1; 2^-32 absolute where it is subnormal there,
    of a maximum of 1), the sums over kv tokens run in fp32 (at most kv / 8 + 64 additions in a row, the
    matrix instruction's eight at a time, doubled for the rescalings), and the result is rounded to bf16."""
    n, qh, D = q.shape
    g = qh // heads
    scale = D ** -0.5 if scale is None else scale
    qd = q.cpu().double()
    kg, vg = float(k_cache.global_[0]), float(v_cache.global_[0])
    pool = k_cache.rows // heads // page
    K = values(k_cache.packed[0], k_cache.scales[0]).view(pool, page, heads, D) if pool else None
    V = values(v_cache.packed[0], v_cache.scales[0]).view(pool, page, heads, D) if pool else None
    out = torch.zeros((n, qh, D), dtype=torch.float64)
    tol = torch.zeros((n, qh, D), dtype=torch.float64)
    lse = torch.full((n, qh), -np.inf, dtype=torch.float64)
    ltol = torch.zeros((n, qh), dtype=torch.float64)
    table, kv_lens = table.cpu(), kv_lens.cpu().tolist()
    cu = list(range(len(kv_lens) + 1)) if cu_q is None else cu_q.cpu().tolist()
    for b, kv in enumerate(kv_lens):
        m = cu[b + 1] - cu[b]
        for i in range(m):
            pos = kv - m + i
            e = min(kv, pos + 1) if causal else kv
            s = max(0, pos - window + 1) if window else 0
            t = torch.arange(s, max(s, e))
            if not len(t):
                continue
            pg = table[b, t // page].long()
            ok = (pg >= 0) & (pg < pool)
            t, pg = t[ok], pg[ok]
            if not len(t):
                continue
            for h in range(heads):
                kk, vv = K[pg, t % page, h] * kg, V[pg, t % page, h] * vg
                x = qd[cu[b] + i, h * g:(h + 1) * g]
                sc = (x @ kk.T) * scale
                S = ((x.abs() @ kk.abs().T) * scale).amax(1)
                S2 = D * x.abs().amax(1) * kk.abs().max() * scale
                z = torch.logsumexp(sc, 1)
                p = torch.exp(sc - z[:, None])
                o = p @ vv
                rows = slice(h * g, (h + 1) * g)
                out[cu[b] + i, rows], lse[cu[b] + i, rows] = o, z
                rel = (D + 4) * STEP * S + STEP * S2
                run = 2 * (len(t) / 8 + 64) * STEP
                tol[cu[b] + i, rows] = (o.abs() * 2.0 ** -8 + (p @ vv.abs()) * (2.0 ** -11 + 2 * rel + run)[:, None]
                                        + 2.0 ** -31 * vv.abs().sum(0) * p.amax(1)[:, None])
                ltol[cu[b] + i, rows] = rel + run + 4 * STEP * (z.abs() + sc.abs().amax(1))
    return out, lse, tol, ltol


def assert_attention(got, lse, ref, what=""):
    out, z, tol, ltol = ref
    d = (got.cpu().double() - out).abs()
    bad = d > tol
    assert not bad.any(), (what, "out", int(bad.sum()), float(d.max()), [int(v) for v in bad.nonzero()[0]])
    if lse is not None:
        lse = lse.cpu().double()
        empty = torch.isinf(z)
        assert torch.equal(empty, torch.isinf(lse)) and bool((lse[empty] < 0).all()), (what, "empty rows")
        d = (lse[~empty] - z[~empty]).abs()
        assert bool((d <= ltol[~empty]).all()), (what, "lse", float((d - ltol[~empty]).max()))


def rotate(x, positions, cos_sin, interleaved):
    """bf16 x [n, heads, D] rotated in fp32 steps as nvfp4_kv_append documents, on the CPU: bf16."""
    rot = cos_sin.shape[1]
    x = x.cpu().float()
    cs = cos_sin.cpu()[positions.cpu().long()][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    out = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out.bfloat16()


def add_rmsnorm(x, residual, weight, eps):
    """(r, y) as mxfp8_add_rmsnorm documents them, on the CPU: bf16."""
    r = x.cpu()
    if residual is not None:
        r = (r.float() + residual.cpu().float()).bfloat16()
    inv = (1.0 / torch.sqrt(r.double().square().mean(1, keepdim=True) + eps)).float()
    w = torch.ones(r.shape[1]) if weight is None else weight.cpu().float()
    return r, (r.float() * inv * w).bfloat16()
