"""The attention half of a decoder layer on NVFP4 / MX operands: what is timed, and its plain form.

Three operators, in the order a serving step runs them:

  norm    the residual's addition, the root-mean-square norm and the MXFP8 encode of its result, as
          the W4A8 projections take it (E4M3 codes, one power-of-two scale per 32)
  append  q and k rotated by position, k and v quantized to NVFP4 and stored in the slots of a paged
          cache that the scheduler chose
  attend  attention of the newest tokens of each sequence over its paged NVFP4 cache: one token each
          (decode), a few (speculation), a chunk (prefill), whole prompts

``run`` with ``own`` false computes them with elementary torch operations in 32 bits (64 for the sum
of squares, whose result sits next to rounding borders), with ``own`` true through the library.
"""
import math
import random

import torch

own = False
DEV = "cuda"

# E2M1 values by code, and a byte's two codes (element 2j in the low nibble)
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1 = GRID + tuple(-v for v in GRID)


def listed():
    return [
        # one user's short chat, one token: the smallest call, latency counts
        dict(name="decode 1 x 700", kind="attend", seqs=1, qh=32, kvh=8, dim=128, page=16, q=1, q_hi=1, kv=700,
             kv_hi=700, window=0, empty=False, lens=1),
        # a busy server's batch of chats of very different lengths, one finished slot among them
        dict(name="decode 64 ragged", kind="attend", seqs=64, qh=32, kvh=8, dim=128, page=16, q=1, q_hi=1, kv=64,
             kv_hi=16384, window=0, empty=True, lens=2),
        # the KV cache configuration of the benchmark (262144 tokens x 4 heads x 256), one request
        dict(name="decode 1 x 262144", kind="attend", seqs=1, qh=32, kvh=4, dim=256, page=64, q=1, q_hi=1, kv=262144,
             kv_hi=262144, window=0, empty=False, lens=3),
        # speculation: five draft tokens a sequence, sliding window layers
        dict(name="draft 24 x 5, window", kind="attend", seqs=24, qh=24, kvh=4, dim=64, page=32, q=5, q_hi=5, kv=3000,
             kv_hi=20000, window=4096, empty=False, lens=4),
        # whole prompts of odd lengths, prefilled together
        dict(name="prompts 7 ragged", kind="attend", seqs=7, qh=32, kvh=8, dim=128, page=16, q=37, q_hi=1900, kv=0,
             kv_hi=0, window=0, empty=False, lens=5),
        # one long prompt
        dict(name="prompt 4096", kind="attend", seqs=1, qh=32, kvh=8, dim=128, page=64, q=4096, q_hi=4096, kv=0,
             kv_hi=0, window=0, empty=False, lens=6),
        # the benchmark's 2048-token chunk on top of a long context
        dict(name="chunk 2048 on 30720", kind="attend", seqs=1, qh=32, kvh=4, dim=256, page=64, q=2048, q_hi=2048,
             kv=30720, kv_hi=30720, window=0, empty=False, lens=7),
        # a decode batch's new tokens
        dict(name="append 64", kind="append", n=64, qh=32, kvh=8, dim=128, rot=128, interleaved=False, page=16,
             far=16384),
        # prefill chunks' new tokens, partial rotation, pairs side by side, far positions
        dict(name="append 16384", kind="append", n=16384, qh=32, kvh=4, dim=256, rot=64, interleaved=True, page=64,
             far=262144),
        # a decode batch at the expert layer's width
        dict(name="norm 64 x 7168", kind="norm", rows=64, cols=7168, residual=True),
        # an odd batch, first layer (nothing to add yet)
        dict(name="norm 777 x 5120", kind="norm", rows=777, cols=5120, residual=False),
        # the prefill batch of the expert layer
        dict(name="norm 16384 x 7168", kind="norm", rows=16384, cols=7168, residual=True),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "draft", "prompts", "chunk", "append", "append", "norm", "norm"])
    if kind == "norm":
        cols = 32 * _log(rng, 4, 400)
        return dict(kind="norm", rows=_log(rng, 1, min(20000, 117440512 // cols)), cols=cols,
                    residual=rng.random() < 0.7)
    dim = rng.choice([64, 128, 256])
    kvh = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if kind == "append":
        qh = kvh * rng.choice([1, 2, 4, 7, 8])
        n = _log(rng, 1, max(2, min(16384, 16384 * 40 * 256 // ((qh + 2 * kvh) * dim))))
        return dict(kind="append", n=n, qh=qh, kvh=kvh, dim=dim, rot=rng.choice([dim, dim, dim // 2, 32]),
                    interleaved=rng.random() < 0.4, page=rng.choice([16, 32, 48, 64, 256]),
                    far=_log(rng, 2 * n, 262144))
    c = dict(kind="attend", page=rng.choice([16, 16, 32, 48, 64, 256]), dim=dim, window=0, empty=rng.random() < 0.3,
             lens=rng.randrange(1 << 30))
    if kind == "decode":
        seqs = _log(rng, 1, 256)
        most = max(64, min(262144, 268435456 // (seqs * kvh * dim)))
        hi = _log(rng, 32, most)
        return dict(c, seqs=seqs, qh=kvh * rng.choice([1, 2, 4, 5, 8, 16]), kvh=kvh, q=1, q_hi=1,
                    kv=_log(rng, 1, hi), kv_hi=hi, window=rng.choice([0, 0, 0, _log(rng, 16, 8192)]))
    if kind == "draft":
        seqs = _log(rng, 1, 48)
        most = max(64, min(65536, 134217728 // (seqs * kvh * dim)))
        hi = _log(rng, 32, most)
        return dict(c, seqs=seqs, qh=kvh * rng.choice([1, 2, 4, 6, 8]), kvh=kvh, q=2, q_hi=rng.choice([3, 5, 8]),
                    kv=_log(rng, 16, hi), kv_hi=hi, window=rng.choice([0, 0, 1024, 4096]))
    kvh = rng.choice([1, 2, 4, 8])
    qh = kvh * rng.choice([1, 4, 5, 8])
    if kind == "prompts":
        seqs = _log(rng, 1, 12)
        hi = _log(rng, 24, max(32, min(4096, int(math.sqrt(4096 * 4096 * 32 / (seqs * qh))))))
        return dict(c, seqs=seqs, qh=qh, kvh=kvh, q=_log(rng, 9, hi), q_hi=hi, kv=0, kv_hi=0,
                    window=rng.choice([0, 0, 512]))
    seqs = _log(rng, 1, 3)
    q_hi = _log(rng, 64, 2048)
    kv_hi = _log(rng, 256, max(512, min(30720, 2048 * 30720 * 32 // (seqs * qh * q_hi * 2))))
    return dict(c, seqs=seqs, qh=qh, kvh=kvh, q=_log(rng, 48, q_hi), q_hi=q_hi, kv=_log(rng, 128, kv_hi),
                kv_hi=kv_hi, window=0)


def _lengths(case):
    """Query tokens and cached tokens (the query's own among them) of each sequence."""
    r = random.Random(case["lens"])
    q, kv = [], []
    for b in range(case["seqs"]):
        nq = _log(r, case["q"], case["q_hi"])
        before = _log(r, case["kv"], case["kv_hi"]) if case["kv_hi"] else 0
        # one token: kv counts it; more: they come on top of the context
        q.append(nq)
        kv.append(before if case["q_hi"] == 1 else before + nq)
    if case["empty"] and case["seqs"] > 1:
        kv[case["seqs"] // 2] = 0  # a slot without a request: its rows have no key
    return q, kv


# ------------------------------------------------------------ the formats --

def _e2m1_code(a):
    """Nearest code of magnitudes a, ties to the even code."""
    c = (a > 0.25).to(torch.uint8)
    for i, edge in enumerate((0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        c += (a >= edge) if i % 2 == 0 else (a > edge)
    return c


def _nvfp4(x, G):
    """bf16 values [..., D] -> (codes uint8 [..., D], block scales fp32 [..., D/16]), static global G."""
    x = x.float().unflatten(-1, (-1, 16))
    s = (x.abs().amax(-1) / (6.0 * G)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    r = torch.where(s > 0, 1.0 / (s * G), torch.zeros_like(s))
    y = x * r[..., None]
    return (_e2m1_code(y.abs()) + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2), s


def _decode(packed, scales, G):
    """fp32 values of NVFP4 bytes: packed [..., D/2], scales [..., D/16]."""
    pair = torch.tensor([(E2M1[b & 15], E2M1[b >> 4]) for b in range(256)], device=packed.device)
    v = pair[packed.int()].flatten(-2).unflatten(-1, (-1, 16))
    return ((v * scales.view(torch.float8_e4m3fn).float()[..., None]) * G).flatten(-2)


# ------------------------------------------------------------ the inputs ---

def _cache(g, rows, dim):
    """An NVFP4 cache tensor of `rows` rows: channels of unequal size, as keys and values have."""
    packed = torch.empty((1, rows, dim // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((1, rows, dim // 16), dtype=torch.uint8, device=DEV)
    channel = torch.exp(0.5 * torch.randn(dim, generator=g, device=DEV))
    G = (7.0 * channel.max() / 2688.0).reshape(1)
    for a in range(0, rows, 1 << 19):
        b = min(rows, a + (1 << 19))
        x = (torch.randn((b - a, dim), generator=g, device=DEV) * channel).bfloat16()
        code, s = _nvfp4(x, G)
        packed[0, a:b] = code[:, ::2] | (code[:, 1::2] << 4)
        scales[0, a:b] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return packed, scales, G


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    if case["kind"] == "norm":
        rows, cols = case["rows"], case["cols"]
        # activations with a few large channels, as residual streams have
        channel = torch.exp(0.7 * torch.randn(cols, generator=g, device=DEV))
        s["x"] = (torch.randn((rows, cols), generator=g, device=DEV) * channel).bfloat16()
        s["residual"] = None
        if case["residual"]:
            s["residual"] = (4 * torch.randn((rows, cols), generator=g, device=DEV) * channel).bfloat16()
        s["weight"] = (1 + 0.3 * torch.randn(cols, generator=g, device=DEV)).bfloat16()
        s["eps"] = 1e-6
        return s
    qh, kvh, dim, page = case["qh"], case["kvh"], case["dim"], case["page"]
    if case["kind"] == "append":
        n, far, rot = case["n"], case["far"], case["rot"]
        # the three parts of one projection's output row
        qkv = torch.randn((n, (qh + 2 * kvh) * dim), generator=g, device=DEV).bfloat16()
        s["q"] = qkv[:, :qh * dim].unflatten(1, (qh, dim))
        s["k"] = qkv[:, qh * dim:(qh + kvh) * dim].unflatten(1, (kvh, dim))
        s["v"] = qkv[:, (qh + kvh) * dim:].unflatten(1, (kvh, dim))
        freq = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angle = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = torch.randint(0, far, (n,), generator=g, device=DEV, dtype=torch.int32)
        pages = -(-n // page) + 3
        slots = torch.randperm(pages, generator=g, device=DEV)[:, None] * page + torch.arange(page, device=DEV)
        s["slots"] = slots.flatten()[:n].clone()
        rows = pages * page * kvh
        G = (5.0 + torch.rand(1, generator=g, device=DEV)) / 2688.0  # calibrated beforehand
        for name in ("k_cache", "v_cache"):
            s[name] = (torch.zeros((1, rows, dim // 2), dtype=torch.uint8, device=DEV),
                       torch.zeros((1, rows, dim // 16), dtype=torch.uint8, device=DEV),
                       G)
        # the cache rows of the new tokens, for reading them back
        s["ids"] = (s["slots"][:, None] * kvh + torch.arange(kvh, device=DEV)).flatten().int()
        return s
    q_lens, kv_lens = _lengths(case)
    n = sum(q_lens)
    s["q"] = (1.5 * torch.randn((n, qh, dim), generator=g, device=DEV)).bfloat16()
    pages = [-(-m // page) for m in kv_lens]
    pool = sum(pages) + 5
    order = torch.randperm(pool, generator=g, device=DEV).int()
    table = torch.full((case["seqs"], max(1, max(pages))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = order[at:at + m]
        at += m
    s["table"], s["max_q"] = table, max(q_lens)
    s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
    cu = torch.zeros(case["seqs"] + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(q_lens, dtype=torch.int32).cumsum(0)
    s["cu_q"] = cu.to(DEV)
    s["k_cache"], s["v_cache"] = _cache(g, pool * page * kvh, dim), _cache(g, pool * page * kvh, dim)
    return s


# ------------------------------------------------------------ plain forms --

def _plain_norm(s):
    r = s["x"]
    if s["residual"] is not None:
        r = (r.float() + s["residual"].float()).bfloat16()
    mean = r.double().square().mean(1, keepdim=True)
    inv = (1.0 / torch.sqrt(mean + s["eps"])).float()
    y = (r.float() * inv * s["weight"].float()).bfloat16().float().unflatten(1, (-1, 32))
    amax = y.abs().amax(-1)
    f, p = torch.frexp(amax)
    e = torch.where(amax > 0, p - 9 + (f > 0.875), 0).clamp(-127, 127)  # 448 = 0.875 * 2^9
    q = torch.ldexp(y, -e[..., None]).to(torch.float8_e4m3fn)
    return {"sum": r, "fp8": q.flatten(1), "exponent": (e + 127).to(torch.uint8)}


def _rotate(x, s):
    half = s["rot"] // 2
    cs = s["cos_sin"][s["positions"].long()][:, None]
    c, sn = cs[..., :half], cs[..., half:]
    x = x.float()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if s["interleaved"] else (x[..., :half], x[..., half:2 * half])
    a, b = a * c - b * sn, b * c + a * sn
    turned = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1).bfloat16()


def _plain_append(s):
    out = {"q": _rotate(s["q"], s)}
    for name, x in (("k", _rotate(s["k"], s)), ("v", s["v"])):
        packed, scales, G = s[name + "_cache"]
        code, sc = _nvfp4(x, G)
        ids = s["ids"].long()
        packed[0, ids] = (code[..., ::2] | (code[..., 1::2] << 4)).flatten(0, 1)
        scales[0, ids] = sc.to(torch.float8_e4m3fn).view(torch.uint8).flatten(0, 1)
        out[name] = _decode(packed[0, ids], scales[0, ids], G).bfloat16()
    return out


def _plain_attend(s):
    qh, kvh, dim, page, seqs, mq = s["qh"], s["kvh"], s["dim"], s["page"], s["seqs"], s["max_q"]
    n = s["q"].shape[0]
    slots = (s["table"].clamp(min=0).long()[:, :, None] * page + torch.arange(page, device=DEV)).flatten(1)
    L = slots.shape[1]
    kv = []
    for packed, scales, G in (s["k_cache"], s["v_cache"]):
        kv.append(_decode(packed.view(-1, kvh, dim // 2)[slots], scales.view(-1, kvh, dim // 16)[slots], G))
    k, v = (t.transpose(1, 2).contiguous() for t in kv)  # [seqs, kvh, L, dim]
    # the queries of each sequence, padded to the longest
    first, count = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(mq, device=DEV)
    at = (first[:, None] + i).clamp(max=n - 1)
    q = s["q"].float()[at].unflatten(2, (kvh, qh // kvh)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (qh // kvh, mq)) * (dim ** -0.5)
    place = s["kv_lens"].long()[:, None] - count[:, None] + i  # each query's own position
    t = torch.arange(L, device=DEV)
    seen = (t <= place[..., None]) & (t < s["kv_lens"][:, None, None])
    if s["window"]:
        seen &= t > place[..., None] - s["window"]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (qh // kvh, mq)) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]
    b = torch.repeat_interleave(torch.arange(seqs, device=DEV), count, output_size=n)
    j = torch.arange(n, device=DEV) - first[b]
    return {"out": o.permute(0, 3, 1, 2, 4)[b, j].flatten(1, 2).bfloat16(),
            "lse": lse.permute(0, 3, 1, 2)[b, j].flatten(1, 2)}


def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend}[s["kind"]](s)
    import precision_moe_gemm_amd as nv
    if s["kind"] == "norm":
        total, _, fp8, e8m0 = nv.mxfp8_add_rmsnorm(s["x"], s["residual"], s["weight"], s["eps"])
        return {"sum": total, "fp8": fp8.view(torch.float8_e4m3fn), "exponent": e8m0}
    kvh = s["kvh"]
    kc, vc = (nv.NVFP4Tensor(p, sc, G, p.shape[1], s["dim"]) for p, sc, G in (s["k_cache"], s["v_cache"]))
    if s["kind"] == "append":
        q = nv.nvfp4_kv_append(s["q"], s["k"], s["v"], s["slots"], kc, vc, s["positions"], s["cos_sin"],
                               interleaved=s["interleaved"])
        return {"q": q, "k": nv.nvfp4_gather_dequantize(kc, s["ids"]), "v": nv.nvfp4_gather_dequantize(vc, s["ids"])}
    out, lse = nv.nvfp4_kv_attention(s["q"], kc, vc, kvh, s["table"], s["kv_lens"], s["page"],
                                     cu_q=s["cu_q"] if s["max_q"] > 1 else None, max_q=s["max_q"],
                                     window=s["window"], return_lse=True)
    return {"out": out, "lse": lse}


def work(case):
    if case["kind"] == "norm":
        n = case["rows"] * case["cols"]
        adds = 2 if case["residual"] else 0  # the residual read; x itself and the sum written come on top
        return {"bytes": n * (2 + adds + 2 + 1) + n // 32 + 2 * case["cols"], "flops": 6 * n}
    qh, kvh, dim = case["qh"], case["kvh"], case["dim"]
    row = dim // 2 + dim // 16  # one NVFP4 row
    if case["kind"] == "append":
        n = case["n"]
        tokens = 2 * qh * dim * 2 + 2 * kvh * (2 * dim + row + 2 * dim)  # and the rows read back in bf16
        return {"bytes": n * (tokens + 4 * case["rot"] + 12), "flops": n * dim * (3 * (qh + kvh) + 4 * 2 * kvh)}
    q_lens, kv_lens = _lengths(case)
    pairs = tokens = 0
    for nq, m in zip(q_lens, kv_lens):
        ends = [min(m, max(0, m - nq + i + 1)) for i in range(nq)]
        lo = [max(0, m - nq + i + 1 - case["window"]) if case["window"] else 0 for i in range(nq)]
        pairs += sum(max(0, e - a) for a, e in zip(lo, ends))
        tokens += max(0, max(ends) - min(lo))
    n = sum(q_lens)
    return {"bytes": n * qh * (4 * dim + 4) + tokens * kvh * 2 * row, "flops": 4 * pairs * qh * dim}


# ------------------------------------------------------------ 64 bits ------

def _exact_row_values(x, G):
    """The values that bf16 x (as float64, [rows, D]) has after NVFP4 quantization, by search over the grids."""
    G = float(G)
    e4m3 = torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device=x.device)
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)

    def nearest(v, values):
        i = torch.bucketize(v, (values[1:] + values[:-1]) / 2)            # a tie: the lower one
        up = (i < len(values) - 1) & (i % 2 == 1)                         # unless that one's code is odd
        mid = ((values[1:] + values[:-1]) / 2)[i.clamp(max=len(values) - 2)]
        return values[torch.where(up & (v == mid), i + 1, i)]

    x = x.reshape(x.shape[0], -1, 16)
    s = nearest((x.abs().amax(2) / (6 * G)).clamp(max=448.0), e4m3)[..., None]
    y = torch.where(s > 0, x / torch.where(s > 0, s, 1.0) / G, 0.0)
    return (torch.sign(x) * nearest(y.abs(), grid) * s * G).reshape(x.shape[0], -1)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["kind"] == "norm":
        x = s["x"].to(f64)
        if s["residual"] is not None:
            x = (x + s["residual"].to(f64)).to(torch.bfloat16).to(f64)
        rms = (x.pow(2).sum(1) / case["cols"] + s["eps"]).sqrt()
        y = (x / rms[:, None] * s["weight"].to(f64)).to(torch.bfloat16).to(f64).reshape(case["rows"], -1, 32)
        top = y.abs().amax(2)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0)).clamp(-127, 127)
        y = y / torch.exp2(e)[..., None]
        # nearest on E4M3's grid: a step is 2^-3 of the value's power of two, 2^-9 at the least
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return {"sum": x, "fp8": (torch.round(y / step) * step).reshape(case["rows"], -1), "exponent": None}
    qh, kvh, dim = case["qh"], case["kvh"], case["dim"]
    if case["kind"] == "append":
        rot, out = case["rot"], {}
        w = s["cos_sin"].to(f64)[s["positions"].long()]
        w = torch.complex(w[:, :rot // 2], w[:, rot // 2:])[:, None]
        for name in ("q", "k"):
            x = s[name].to(f64).clone()
            even = list(range(0, rot, 2)) if case["interleaved"] else list(range(rot // 2))
            odd = [i + 1 for i in even] if case["interleaved"] else [i + rot // 2 for i in even]
            z = torch.complex(x[..., even], x[..., odd]) * w
            x[..., even], x[..., odd] = z.real, z.imag
            out[name] = x
        out["k"] = _exact_row_values(out["k"].to(torch.bfloat16).to(f64).reshape(-1, dim), s["k_cache"][2])
        out["v"] = _exact_row_values(s["v"].to(f64).reshape(-1, dim), s["v_cache"][2])
        return out
    q_lens, kv_lens = _lengths(case)
    if max(a * b for a, b in zip(q_lens, kv_lens)) * qh > 1 << 31:
        return None
    value = torch.tensor(E2M1, dtype=f64, device=DEV)
    out, lse, at = [], [], 0
    for b, (nq, m) in enumerate(zip(q_lens, kv_lens)):
        t = torch.arange(m, device=DEV)
        row = s["table"][b].long()[t // case["page"]] * case["page"] + t % case["page"]
        kv = []
        for packed, scales, G in (s["k_cache"], s["v_cache"]):
            p = packed.view(-1, kvh, dim // 2)[row]
            x = torch.empty((m, kvh, dim), dtype=f64, device=DEV)
            x[..., ::2], x[..., 1::2] = value[(p & 15).long()], value[(p >> 4).long()]
            sc = scales.view(-1, kvh, dim // 16)[row].view(torch.float8_e4m3fn).to(f64)
            kv.append(x * sc.repeat_interleave(16, 2) * float(G))
        q = s["q"][at:at + nq].to(f64)
        at += nq
        pos = torch.arange(nq, device=DEV) + (m - nq)
        hide = t[None] > pos[:, None]
        if case["window"]:
            hide = hide | (t[None] <= pos[:, None] - case["window"])
        o = torch.zeros((nq, qh, dim), dtype=f64, device=DEV)
        z = torch.full((nq, qh), -math.inf, dtype=f64, device=DEV)
        for h in range(qh if m else 0):
            x = (q[:, h] @ kv[0][:, h // (qh // kvh)].T) / math.sqrt(dim)
            x[hide] = -math.inf
            z[:, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - torch.where(z[:, h:h + 1] > -math.inf, z[:, h:h + 1], 0.0))
            o[:, h] = p @ kv[1][:, h // (qh // kvh)]
        out.append(o)
        lse.append(z)
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
