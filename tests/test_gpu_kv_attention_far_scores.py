"""GPU: nvfp4_kv_attention where scores lie far from zero, from 2^20 to fp32's end, against the formula in 64 bits.

Every row has one channel that differs from zero, so a score is one product, exact but for the roundings of
its factors.  Keys differ in that channel by steps of 0.5 and more, so at these sizes the tokens with a row's
largest score take all the weight, evenly: equal keys have equal errors.  Bounds: the output's rounding to
bf16 (2^-8 of it), the weights' to f16 (2^-11 of the mean magnitude) and the sums' (at most 2500 / 8 + 64
additions in a row, doubled for the rescalings: below 2^-14).  A score has 5 roundings (row factor, product,
the base of the exponential and back, the subtraction of the maximum) and lse 4 more (the sum, its logarithm,
the product with ln 2, the addition): STEPS, of the largest score and the logarithm's size, doubled.  Where
scores lie near zero the weights differ by as much again.  A weight below 2^-14 of 2^7 times its row's largest is
subnormal in f16, off by at most 2^-25 there: 2^-32 of the largest for every token, doubled, which counts in
elements where the heavy tokens' values are zero."""
import math

import pytest
import torch

from tests.attn_check import values
from tests.gpu_util import step
from tests.test_gpu_kv_attention import DEV, call, make_case

pytestmark = pytest.mark.gpu
STEPS = 9 * 2.0 ** -24
KEYS = [0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # E2M1 magnitudes: exact under a block scale of 1


def place_keys(c, keys):
    """keys float [seqs, tokens] in channel 3 of every head; all other channels zero, scales 1, global 1."""
    D, heads, page = c["q"].shape[2], c["heads"], c["page"]
    kc = c["k_cache"]
    codes = torch.zeros((keys.shape[0], keys.shape[1], heads, D // 2), dtype=torch.uint8)
    grid = torch.tensor([0.0] + KEYS)
    code = (keys.abs()[..., None] == grid).float().argmax(-1) + 8 * (keys < 0)
    codes[..., 1] = (code.to(torch.uint8) << 4)[..., None]  # element 3: the high nibble of byte 1
    packed, scales = kc.packed.view(-1, page, heads, D // 2), kc.scales.view(-1, page, heads, D // 16)
    for b, m in enumerate(c["kv_lens"].tolist()):
        t = torch.arange(m)
        pg = c["table"][b].cpu()[t // page].long().to(DEV)
        packed[pg, (t % page).to(DEV)] = codes[b, :m].to(DEV)
        scales[pg, (t % page).to(DEV)] = 0x38
    kc.global_.fill_(1.0)


def reference(c, keys, scale, spread):
    """(out, lse, tolerances) in 64 bits; spread: scores near zero, whose weights differ by their roundings."""
    n, qh, D = c["q"].shape
    heads, page = c["heads"], c["page"]
    vc = c["v_cache"]
    V = values(vc.packed[0], vc.scales[0]).view(-1, page, heads, D) * float(vc.global_[0])
    cu = c["cu_q"].tolist() if c["cu_q"] is not None else list(range(n + 1))
    q = c["q"].cpu().double()[..., 3].unflatten(1, (heads, -1))
    out, lse = torch.zeros((n, heads, qh // heads, D), dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b, m in enumerate(c["kv_lens"].tolist()):
        t, rows = torch.arange(m), slice(cu[b], cu[b + 1])
        hide = t > torch.arange(m - cu[b + 1] + cu[b], m)[:, None]
        vb = V[c["table"][b].cpu()[t // page].long(), t % page]
        for h in range(heads):
            s = q[rows, h, :, None] * keys[b, :m].double() * scale
            s = s.masked_fill(hide[:, None], -math.inf)
            most = s.masked_fill(hide[:, None], 0).abs().amax(-1)
            z = torch.logsumexp(s, -1)
            w = torch.softmax(s, -1)  # (past 2^53 the logarithm of their number is lost in z)
            size = w @ vb[:, h].abs()
            out[rows, h], lse[rows, h] = w @ vb[:, h], z
            rel = 2.0 ** -11 + 2.0 ** -14 + (2 * STEPS * most[..., None] if spread else 0)
            tol[rows, h] = (out[rows, h].abs() * 2.0 ** -8 + size * rel
                            + 2.0 ** -31 * w.amax(-1, keepdim=True) * vb[:, h].abs().sum(0))
            ltol[rows, h] = 2 * STEPS * (most + math.log(m) + 10)
    return out.flatten(1, 2), lse.flatten(1), tol.flatten(1, 2), ltol.flatten(1)


def check(c, keys, scale, what, spread=False):
    step(what)
    out, lse = call(c, scale=scale)
    torch.cuda.synchronize()
    wo, wl, tol, ltol = reference(c, keys, float(torch.tensor(scale, dtype=torch.float32)), spread)
    past = wl.abs() > 2.35e38  # (fp32's largest value times ln 2: scores past it count as it)
    assert out.isfinite().all() and lse.isfinite().all(), what
    assert (lse.cpu()[past].sign() == wl[past].sign()).all(), what
    bad = ~((out.cpu().double() - wo).abs() <= tol) & ~past[..., None]
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())
    bad = ~((lse.cpu().double() - wl).abs() <= ltol) & ~past
    assert not bad.any(), (what, "lse", int(bad.sum()), bad.nonzero()[0].tolist())


# (query rows per KV head: 4, 20, 80 and 360)
CALLS = [([1, 1, 1], [1, 40, 1500], True, "shares"), ([1, 1], [90, 300], True, "one launch"),
         ([5, 3], [90, 1300], False, "row tiles of 32"), ([20, 3], [2500, 70], False, "128-row tiles, split"),
         ([90, 2], [300, 70], False, "256-row tiles"), ([90, 2], [2500, 70], False, "256-row tiles, split")]


def random_keys(c, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.tensor(KEYS)[torch.randint(0, 7, (len(c["kv_lens"]), int(c["kv_lens"].max())), generator=g)]


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,decode,what", CALLS)
def test_far_scores(q_lens, kv_lens, decode, what, D, order):
    c = make_case(q_lens, kv_lens, 2, 4, D, 16, seed=D, decode=decode)
    keys = random_keys(c, len(order))
    if order != "mixed":
        keys = keys.sort(1, descending=order == "falling").values
    place_keys(c, keys)
    n, qh, _ = c["q"].shape
    g = torch.Generator().manual_seed(5)
    for e in (20, 23, 25, 28, 40, 60, 100, 123):
        sign = torch.where(torch.rand((n, qh), generator=g) < 0.5, -1.0, 1.0)
        size = (1 + torch.randint(0, 128, (n, qh), generator=g) / 128) * 2.0 ** e
        c["q"].zero_()
        c["q"][..., 3] = (sign * size).bfloat16().to(DEV)
        check(c, keys, 1.0, f"scores of 2^{e}, {what}, D = {D}, {order}")


@pytest.mark.parametrize("q_lens,kv_lens,decode,what", CALLS)
def test_scores_past_fp32(q_lens, kv_lens, decode, what):
    """They count as the largest that fp32 holds: nothing becomes NaN or a row that sees nothing."""
    c = make_case(q_lens, kv_lens, 2, 4, 128, 16, seed=1, decode=decode)
    keys = torch.full((len(kv_lens), max(kv_lens)), 6.0)
    keys[:, ::2] = 0.5
    place_keys(c, keys)
    top = 3.3895313892515355e38  # the largest bf16
    for value in (top, -top):
        c["q"].zero_()
        c["q"][..., 3] = value
        for scale in (1.0, 100.0, 2.9e38):
            step(f"queries of {value}, scale {scale}, {what}")
            out, lse = call(c, scale=scale)
            torch.cuda.synchronize()
            assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all(), (value, scale)
            assert ((lse > 0) == (value > 0)).all()


@pytest.mark.parametrize("scale,q,glob", [(2.9e38, 2.0 ** -120, 1.0), (2.9e38, 1.0, 2.0 ** -120),
                                          (1e-37, 2.0 ** 100, 2.0 ** 20), (1e-37, 2.0 ** 127, 1.0),
                                          (3e-30, 2.0 ** -10, 2.0 ** 105)])
def test_factors_whose_product_alone_is_ordinary(scale, q, glob):
    """The scale, a row's size and the keys' global at the ends of their ranges."""
    for q_lens, kv_lens, decode, what in CALLS:
        c = make_case(q_lens, kv_lens, 1, 4, 64, 16, seed=2, decode=decode)
        keys = random_keys(c, 3)
        place_keys(c, keys)
        c["k_cache"].global_.fill_(glob)
        c["q"].zero_()
        c["q"][..., 3] = q
        check(c, keys * glob, scale, f"scale {scale}, q {q}, global {glob}, {what}", spread=True)


@pytest.mark.parametrize("e,scale", [(10, 0.125), (60, 0.125), (110, 1.0), (127, 1.0), (127, 100.0)])
@pytest.mark.parametrize("q_lens,kv_lens,decode,what", CALLS)
def test_a_maximum_of_zero_before_far_scores(q_lens, kv_lens, decode, what, e, scale):
    """Keys of zero first: a maximum of 0 under a factor of up to 2^134, then scores that leave it behind or stay
    far below it."""
    c = make_case(q_lens, kv_lens, 2, 4, 128, 16, seed=e, decode=decode)
    keys = random_keys(c, 4)
    keys[:, :max(kv_lens) * 2 // 3] = 0
    keys[:, 0] = 0
    place_keys(c, keys)
    g = torch.Generator().manual_seed(6)
    sign = torch.where(torch.rand(c["q"].shape[:2], generator=g) < 0.5, -1.0, 1.0)
    c["q"].zero_()
    c["q"][..., 3] = (sign * 2.0 ** e).to(DEV)
    check(c, keys, scale, f"zeros before scores of 2^{e}, scale {scale}, {what}")
