"""The attention half of a decoder layer as a serving loop runs it: norm -> W4A8 projection of q, k
and v -> append -> attention -> output projection, a prefilled prompt and then tokens one by one.

Each step is checked against the separate entry points or the formula on that step's own inputs."""
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.attn_check import add_rmsnorm, assert_attention, attention, rotate
from tests.gpu_util import step

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, QH, KVH, D, PAGE = 512, 8, 2, 128, 16


class Block:
    def __init__(self, seqs, pages_per_seq):
        g = torch.Generator().manual_seed(1)
        width = (QH + 2 * KVH) * D
        self.norm_w = (1 + 0.2 * torch.randn(H, generator=g)).bfloat16().to(DEV)
        self.wqkv = nv.mxfp4_quantize((torch.randn((width, H), generator=g) * H ** -0.5).bfloat16().to(DEV))
        self.wo = nv.mxfp4_quantize((torch.randn((H, QH * D), generator=g) * (QH * D) ** -0.5).bfloat16().to(DEV))
        freq = 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        a = torch.arange(4096, dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().to(DEV)
        pool = seqs * pages_per_seq + 2
        self.caches = []
        for _ in range(2):
            t = nv.NVFP4Tensor.empty(pool * PAGE * KVH, D, 1, DEV)
            t.packed.fill_(0xFF)
            t.scales.fill_(0x7F)
            t.global_.fill_(6.0 / 2688)
            self.caches.append(t)
        self.table = torch.randperm(pool, generator=g)[:seqs * pages_per_seq].view(seqs, -1).int().to(DEV)

    def slots(self, seq, pos):
        return (self.table[seq, pos // PAGE].long() * PAGE + pos % PAGE).contiguous()

    def run(self, x, residual, positions, slots, kv_lens, cu_q, max_q):
        n = x.shape[0]
        self.r, self.y, fp8, e8 = nv.mxfp8_add_rmsnorm(x, residual, self.norm_w, want_y=True)
        qkv = nv.mx_gemm_w4a8(fp8, e8, *self.wqkv, dtype=torch.bfloat16)
        q = qkv[:, :QH * D].unflatten(1, (QH, D))
        k = qkv[:, QH * D:(QH + KVH) * D].unflatten(1, (KVH, D))
        v = qkv[:, (QH + KVH) * D:].unflatten(1, (KVH, D))
        self.qkv = (q, k, v)
        self.fp8 = (fp8, e8)
        self.q = nv.nvfp4_kv_append(q, k, v, slots, *self.caches, positions, self.cos_sin)
        self.o, self.lse = nv.nvfp4_kv_attention(self.q, *self.caches, KVH, self.table, kv_lens, PAGE, cu_q=cu_q,
                                                 max_q=max_q, return_lse=True)
        of, oe = nv.mxfp8_quantize(self.o.reshape(n, -1))
        return nv.mx_gemm_w4a8(of, oe, *self.wo, dtype=torch.bfloat16)

    def check(self, x, residual, positions, slots, kv_lens, cu_q):
        r, y = add_rmsnorm(x, residual, self.norm_w, 1e-6)
        assert torch.equal(self.r.cpu(), r) and torch.equal(self.y.cpu(), y)
        for got, want in zip(self.fp8, nv.mxfp8_quantize(y.to(DEV))):
            assert torch.equal(got, want)
        q, k, v = self.qkv
        assert torch.equal(self.q.cpu(), rotate(q, positions, self.cos_sin, False))
        for x, cache in ((rotate(k, positions, self.cos_sin, False).to(DEV), self.caches[0]), (v, self.caches[1])):
            want = nv.nvfp4_quantize(x.reshape(-1, D).contiguous(), static_global=cache.global_)
            assert torch.equal(cache.packed.view(-1, KVH, D // 2)[slots].view(-1, D // 2), want.packed[0])
            assert torch.equal(cache.scales.view(-1, KVH, D // 16)[slots].view(-1, D // 16), want.scales[0])
        assert_attention(self.o, self.lse, attention(self.q, *self.caches, KVH, self.table, kv_lens, PAGE, cu_q=cu_q))


def test_prefill_then_decode():
    lens = [50, 7, 129]
    blk = Block(3, 10)
    g = torch.Generator().manual_seed(2)
    n = sum(lens)
    x, res = (torch.randn((n, H), generator=g).bfloat16().to(DEV) for _ in range(2))
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(lens)).to(DEV)
    pos = torch.cat([torch.arange(m) for m in lens]).int().to(DEV)
    cu = torch.tensor([0, 50, 57, 186], dtype=torch.int32, device=DEV)
    kv = torch.tensor(lens, dtype=torch.int32, device=DEV)
    step("prefill")
    slots = blk.slots(seq, pos.long())
    out = blk.run(x, res, pos, slots, kv, cu, max(lens))
    torch.cuda.synchronize()
    blk.check(x, res, pos, slots, kv, cu)
    assert torch.isfinite(out.float()).all() and nv.nvfp4_get_error() == 0

    # decode: the loop body captured once, its inputs updated between replays; each replay equals the eager pass
    xd, rd = (torch.randn((3, H), generator=g).bfloat16().to(DEV) for _ in range(2))
    pos, kv = kv.clone(), kv + 1
    slots = blk.slots(torch.arange(3, device=DEV), pos.long())
    step("decode, eager")
    blk.run(xd, rd, pos, slots, kv, None, 1)
    torch.cuda.synchronize()
    blk.check(xd, rd, pos, slots, kv, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = blk.run(xd, rd, pos, slots, kv, None, 1)
    r, lse, o = blk.r, blk.lse, blk.o
    for rep in range(12):
        xd.copy_(torch.randn((3, H), generator=g).bfloat16())
        pos.add_(1)
        kv.add_(1)
        slots.copy_(blk.slots(torch.arange(3, device=DEV), pos.long()))
        torch.cuda.synchronize()
        step(f"decode, replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        replayed = got.clone(), o.clone(), lse.clone()
        eager = blk.run(xd, rd, pos, slots, kv, None, 1)
        for a, b in zip(replayed, (eager, blk.o, blk.lse)):
            assert torch.equal(a, b), rep
    blk.check(xd, rd, pos, slots, kv, None)
    assert nv.nvfp4_get_error() == 0
