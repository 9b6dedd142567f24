"""GPU parity: nvfp4_kv_append against the rotation in fp32 steps and the oracle's quantization, byte for byte."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from precision_moe_gemm_amd import synth
from tests.attn_check import rotate
from tests.gpu_util import step, u8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def table(far, rot):
    freq = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(far, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def make(n, qh, heads, D, rot, page=16, far=3000, seed=0, G=(0.003, 0.0017)):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((n, (qh + 2 * heads) * D), generator=g).bfloat16().to(DEV)
    q = qkv[:, :qh * D].unflatten(1, (qh, D))
    k = qkv[:, qh * D:(qh + heads) * D].unflatten(1, (heads, D))
    v = qkv[:, (qh + heads) * D:].unflatten(1, (heads, D))
    pages = -(-n // page) + 2
    caches = []
    for x in G:
        t = nv.NVFP4Tensor.empty(pages * page * heads, D, 1, DEV)
        t.packed.fill_(0xAB)
        t.scales.fill_(0xCD)
        t.global_.fill_(x)
        caches.append(t)
    slots = torch.randperm(pages * page, generator=g)[:n].to(DEV)
    pos = torch.randint(0, far, (n,), generator=g).int().to(DEV)
    return dict(q=q, k=k, v=v, slots=slots, k_cache=caches[0], v_cache=caches[1], positions=pos,
                cos_sin=table(far, rot).to(DEV) if rot else None)


def check(orc, c, interleaved, q, kept=None):
    n, heads, D = c["k"].shape
    turn = (lambda x: rotate(x, c["positions"].clamp(0, c["cos_sin"].shape[0] - 1), c["cos_sin"], interleaved)) \
        if c["cos_sin"] is not None else (lambda x: x.cpu())
    kept = list(range(n)) if kept is None else kept
    if q is not None:
        assert torch.equal(q.cpu().view(torch.int16), turn(c["q"]).view(torch.int16))
    for name, x, cache in (("k", turn(c["k"]), c["k_cache"]), ("v", c["v"].cpu(), c["v_cache"])):
        ref = orc.quantize(np.ascontiguousarray(synth.bits(x[kept].contiguous()).reshape(-1, D)),
                           static_G=float(cache.global_[0]))
        packed = np.full((cache.rows // heads, heads, D // 2), 0xAB, np.uint8)
        scales = np.full((cache.rows // heads, heads, D // 16), 0xCD, np.uint8)
        at = c["slots"].cpu().numpy()[kept]
        packed[at] = ref.packed.reshape(-1, heads, D // 2)
        scales[at] = ref.scales.reshape(-1, heads, D // 16)
        np.testing.assert_array_equal(u8(cache.scales)[0].reshape(scales.shape), scales, err_msg=name)
        np.testing.assert_array_equal(u8(cache.packed)[0].reshape(packed.shape), packed, err_msg=name)


def call(c, interleaved=False, **kw):
    return nv.nvfp4_kv_append(c["q"], c["k"], c["v"], c["slots"], c["k_cache"], c["v_cache"], c["positions"],
                              c["cos_sin"], interleaved=interleaved, **kw)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 96), (256, 256), (256, 64),
                                   (96, 96), (96, 32), (32, 32), (160, 64), (512, 512)])
def test_bytes(orc, D, rot, interleaved):
    c = make(37, 6, 3, D, rot, seed=D + rot)
    step(f"append D={D} rot={rot} interleaved={interleaved}")
    q = call(c, interleaved)
    torch.cuda.synchronize()
    check(orc, c, interleaved, q)
    assert nv.nvfp4_get_error() == 0


@pytest.mark.parametrize("n", [1, 2, 63, 64, 1000, 5000])
@pytest.mark.parametrize("qh,heads", [(1, 1), (32, 8), (5, 5)])
def test_batches(orc, n, qh, heads):
    c = make(n, qh, heads, 128, 128, seed=n)
    step(f"append n={n} heads {qh}/{heads}")
    check(orc, c, False, call(c))


def test_without_rotation_and_without_parts(orc):
    c = make(19, 4, 2, 128, 0, seed=3)
    q = call(c)
    assert torch.equal(q, c["q"])
    check(orc, c, False, None)
    d = make(19, 4, 2, 128, 128, seed=4)
    nv.nvfp4_kv_append(None, d["k"], None, d["slots"], d["k_cache"], d["v_cache"], d["positions"], d["cos_sin"])
    assert (d["v_cache"].packed == 0xAB).all() and (d["v_cache"].scales == 0xCD).all()
    nv.nvfp4_kv_append(None, None, d["v"], d["slots"], d["k_cache"], d["v_cache"])
    check(orc, d, False, None)
    only = nv.nvfp4_kv_append(d["q"], None, None, d["slots"], d["k_cache"], d["v_cache"], d["positions"], d["cos_sin"],
                              heads=2)
    check(orc, d, False, only)


@pytest.mark.parametrize("interleaved", [False, True])
def test_q_in_place(orc, interleaved):
    c = make(300, 8, 2, 256, 256, seed=5)
    want = call(c, interleaved)
    before = c["q"].clone()
    got = call(c, interleaved, q_out=c["q"])
    assert torch.equal(got, want) and got.data_ptr() == c["q"].data_ptr()
    c["q"] = before
    check(orc, c, interleaved, got)


def test_equals_kv_quant_of_the_rotated_k():
    c = make(64, 4, 4, 256, 256, page=64, seed=6)
    c["slots"] = torch.arange(64, device=DEV) + 64
    call(c)
    k = rotate(c["k"], c["positions"], c["cos_sin"], False).to(DEV)
    other = [nv.NVFP4Tensor.empty(t.rows, 256, 1, DEV) for t in (c["k_cache"], c["v_cache"])]
    for o, t in zip(other, (c["k_cache"], c["v_cache"])):
        o.packed.fill_(0xAB)
        o.scales.fill_(0xCD)
        o.global_.copy_(t.global_)
    nv.nvfp4_kv_quant(k, c["v"].contiguous(), 64, other[0], other[1], 4)
    for o, t in zip(other, (c["k_cache"], c["v_cache"])):
        assert torch.equal(o.packed, t.packed) and torch.equal(o.scales, t.scales)


def test_padding_and_bad_slots_and_positions(orc):
    c = make(50, 4, 2, 64, 64, seed=7)
    c["slots"][3] = -1
    c["slots"][20] = -(1 << 40)
    c["positions"][20] = -9          # a padding token's position is nobody's: its q row alone is zero
    step("padding")
    q = call(c)
    assert nv.nvfp4_get_error() == 0
    kept = [i for i in range(50) if i not in (3, 20)]
    assert (q[20] == 0).all()
    want = rotate(c["q"], c["positions"].clamp(min=0), c["cos_sin"], False)
    assert torch.equal(q.cpu()[kept + [3]], want[kept + [3]])
    check(orc, c, False, None, kept)
    d = make(50, 4, 2, 64, 64, seed=8)
    d["slots"][4] = 1 << 40
    d["positions"][11] = 3000
    step("slots and positions out of range")
    q = call(d)
    assert nv.nvfp4_get_error() == 3 and nv.nvfp4_get_error() == 0
    assert (q[11] == 0).all()
    check(orc, d, False, None, [i for i in range(50) if i not in (4, 11)])


def test_the_same_slot_twice_touches_no_other(orc):
    c = make(20, 2, 2, 128, 128, seed=9)
    c["slots"][7] = c["slots"][12]
    call(c)
    torch.cuda.synchronize()
    at = int(c["slots"][7])
    for t in (c["k_cache"], c["v_cache"]):
        t.packed.view(-1, 2, 64)[at] = 0
        t.scales.view(-1, 2, 8)[at] = 0
    d = make(20, 2, 2, 128, 128, seed=9)
    keep = torch.tensor([i for i in range(20) if i not in (7, 12)], device=DEV)
    nv.nvfp4_kv_append(None, d["k"][keep], d["v"][keep], c["slots"][keep], d["k_cache"], d["v_cache"],
                       d["positions"][keep], d["cos_sin"])
    for t, u in ((c["k_cache"], d["k_cache"]), (c["v_cache"], d["v_cache"])):
        u.packed.view(-1, 2, 64)[at] = 0
        u.scales.view(-1, 2, 8)[at] = 0
        assert torch.equal(t.packed, u.packed) and torch.equal(t.scales, u.scales)


def test_empty_batch_and_refusals():
    c = make(4, 2, 2, 64, 64, seed=10)
    e = dict(c, q=c["q"][:0], k=c["k"][:0], v=c["v"][:0], slots=c["slots"][:0], positions=c["positions"][:0])
    assert call(e).shape == (0, 2, 64)
    assert (c["k_cache"].packed == 0xAB).all()
    for name, v in (("q", c["q"].float()), ("k", c["k"][:2]), ("slots", c["slots"].int()),
                    ("positions", c["positions"].long()), ("cos_sin", c["cos_sin"].double()),
                    ("v", c["v"].cpu()), ("positions", None)):
        with pytest.raises((ValueError, AttributeError)):
            call(dict(c, **{name: v}))
    with pytest.raises(nv.NVFP4Error):
        call(dict(c, cos_sin=c["cos_sin"][:, :48].contiguous()))


def test_graph_replays(orc):
    c = make(33, 4, 2, 128, 128, seed=11)
    call(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = call(c)
    for rep in range(3):
        c["positions"].add_(17)
        for t in (c["k_cache"], c["v_cache"]):
            t.packed.fill_(0xAB)
            t.scales.fill_(0xCD)
        torch.cuda.synchronize()
        step(f"append replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        # positions that passed the table's end: documented as stored nowhere, q rows of zeros
        kept = (c["positions"] < c["cos_sin"].shape[0]).nonzero().flatten().tolist()
        want = rotate(c["q"], c["positions"].clamp(max=c["cos_sin"].shape[0] - 1), c["cos_sin"], False)
        want[[i for i in range(33) if i not in kept]] = 0
        assert torch.equal(q.cpu().view(torch.int16), want.view(torch.int16)), rep
        check(orc, c, False, None, kept)
        assert nv.nvfp4_get_error() == (0 if len(kept) == 33 else 3)
