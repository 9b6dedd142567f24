"""GPU parity: what a single weight can be.  Rows of q with a NaN or an infinity, and log-sum-exps that are not
those of the rows."""
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.attn_check import STEP, values
from tests.cache_check import causal_seen, received
from tests.gpu_util import step
from tests.test_gpu_kv_weights import DEV, agree, call, make, with_lse

pytestmark = pytest.mark.gpu
Q, KV = [6, 40, 1], [90, 300, 70]
# row of q, query head, element, value
ODD = [(1, 0, 3, float("nan")), (4, 2, 0, float("inf")), (20, 3, 100, float("inf")), (21, 1, 0, -float("inf")),
       (46, 1, 17, -float("inf"))]


def make_odd(D):
    c = with_lse(make(Q, KV, 2, 2, D, 16, seed=41))
    c["fine"] = c["lse"].clone()
    for row, head, e, v in ODD:
        c["q"][row, head, e % D] = v
    return c


def reference(c):
    return received(c["q"], c["lse"], c["k_cache"], 2, c["table"], c["kv_lens"], 16, c["before"], cu_q=c["cu_q"])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("attention_max_q", [1, 200])
def test_rows_that_are_not_finite_add_nothing(D, attention_max_q):
    """With what the attention returns for them, by rows and by tiles."""
    c = make_odd(D)
    own, c["max_q"] = c["max_q"], attention_max_q
    with_lse(c)
    c["max_q"] = own
    finite = torch.ones_like(c["lse"], dtype=torch.bool)
    for row, head, _, _ in ODD:
        finite[row, head] = False
    assert torch.equal(torch.isfinite(c["lse"]), finite)
    ref = reference(c)
    for max_q in (1, 16, 32, 200):
        step(f"rows that are not finite, D={D} max_q={max_q}")
        agree(call(c, max_q=max_q), ref, 7.0, f"D={D} max_q={max_q}")
    assert nv.nvfp4_get_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 16, 32, 200])
def test_infinite_scores_under_a_finite_lse(D, max_q):
    """0 or 1 by their sign, and 0 where they are NaN (an element of K is zero).  Each one more adds to the sum's bound
    what cache_check.received says of sums: R + 4 steps and 2 of it, R = m * 2 rows."""
    c = make_odd(D)
    c["lse"] = c["fine"]
    want, tol, written = reference(c)
    pool = c["k_cache"].rows // 2 // 16
    K = values(c["k_cache"].packed[0], c["k_cache"].scales[0]).view(pool, 16, 2, D)
    first = 0
    for b, (m, kv) in enumerate(zip(Q, KV)):
        for i, seen in enumerate(causal_seen(m, kv, True, 0)):
            for row, head, e, v in ODD:
                if row == first + i:
                    t = torch.tensor(seen)
                    page = c["table"][b].cpu().long()[t // 16]
                    one = (v * K[page, t % 16, head // 2, e % D] > 0).double()
                    want[head // 2, page * 16 + t % 16] += one
                    tol[head // 2, page * 16 + t % 16] += (2 * m + 6) * STEP * one
        first += m
    step(f"infinite scores, D={D} max_q={max_q}")
    agree(call(c, max_q=max_q), (want, tol, written), 7.0, f"D={D} max_q={max_q}")
    assert nv.nvfp4_get_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 16, 32, 200])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 33), (False, 0)])
def test_a_weight_past_one_counts_as_one(D, max_q, causal, window):
    """Log-sum-exps lowered by 300: every weight is one, and a token's sum the number of rows and heads that see it
    (whole numbers, so equal)."""
    c = with_lse(make([1, 30], [90, 200], 2, 3, D, 16, seed=43), causal=causal, window=window)
    c["lse"] -= 300.0
    step(f"weights past one, D={D} max_q={max_q} causal={causal} window={window}")
    out = call(c, weights=None, out=torch.full_like(c["before"], 7.0), max_q=max_q, causal=causal, window=window)
    torch.cuda.synchronize()
    want = torch.full_like(out, 7.0).cpu()
    for b, (m, kv) in enumerate(zip([1, 30], [90, 200])):
        n = torch.zeros(kv)
        for seen in causal_seen(m, kv, causal, window):
            n[seen] += 3
        t = torch.arange(kv)
        want[:, c["table"][b].cpu().long()[t // 16] * 16 + t % 16] = n
    assert torch.equal(out.cpu(), want)
