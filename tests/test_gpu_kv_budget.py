"""Trees of drafts on a cache of bounded length, as a serving loop runs them: prompts are appended, attended and
weighed; then step by step a tree of drafts is appended and attended, its accepted path is moved together and weighed,
and sequences past their budget give up tokens.

Each call is checked against its formula on that step's own inputs, and the cache's rows against a list of what
every KV head of a sequence should hold."""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.attn_check import assert_attention, attention
from tests.cache_check import chosen, mask_of, received, tree_attention
from tests.gpu_util import step
from tests.test_gpu_kv_weights import agree

pytestmark = pytest.mark.gpu
DEV = "cuda"
QH, KVH, PAGE = 8, 2, 16


class Layer:
    def __init__(self, seqs, pages, D, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.r = np.random.default_rng(seed)
        self.D, self.seqs = D, seqs
        pool = seqs * pages + 2
        self.caches = []
        for _ in range(2):
            t = nv.NVFP4Tensor.empty(pool * PAGE * KVH, D, 1, DEV)
            t.packed.fill_(0xFF)
            t.scales.fill_(0x7F)
            t.global_.fill_(6.0 / 2688)
            self.caches.append(t)
        self.table = torch.randperm(pool, generator=self.g)[:seqs * pages].view(seqs, pages).int().to(DEV)
        self.weights = torch.full((KVH, pool * PAGE), float("nan"), device=DEV)  # nothing unwritten may be read
        self.positions = torch.full((KVH, pool * PAGE), -1, dtype=torch.int32, device=DEV)
        freq = 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        a = torch.arange(1024, dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().to(DEV)
        self.lens, self.ends = [0] * seqs, [0] * seqs  # cached tokens, positions
        self.held = [[[] for _ in range(KVH)] for _ in range(seqs)]  # (position, bytes) by place

    def slots(self, b, places):
        places = torch.as_tensor(places, dtype=torch.long)
        return self.table[b].cpu().long()[places // PAGE] * PAGE + places % PAGE

    def append(self, b_places, b_positions):
        """New tokens of every sequence at the given places and positions: their rotated queries."""
        n = sum(len(p) for p in b_places)
        qkv = torch.randn((n, (QH + 2 * KVH) * self.D), generator=self.g).bfloat16().to(DEV)
        q, k, v = (x.unflatten(1, (-1, self.D)) for x in qkv.split([QH * self.D, KVH * self.D, KVH * self.D], 1))
        slots = torch.cat([self.slots(b, p) for b, p in enumerate(b_places)])
        pos = torch.tensor([x for p in b_positions for x in p], dtype=torch.int32)
        q = nv.nvfp4_kv_append(q, k, v, slots.to(DEV), *self.caches, pos.to(DEV), self.cos_sin)
        self.positions[:, slots.to(DEV)] = pos.to(DEV)
        for b, (places, where) in enumerate(zip(b_places, b_positions)):
            for p, x in zip(places, where):
                for h in range(KVH):
                    assert len(self.held[b][h]) == p
                    self.held[b][h].append((x, self.row(b, h, p)))
        return q

    def row(self, b, h, place):
        r = int(self.slots(b, [place])[0]) * KVH + h
        return b"".join(t.cpu().numpy().tobytes() for c in self.caches for t in (c.packed[0, r], c.scales[0, r]))

    def call_args(self):
        return KVH, self.table, torch.tensor(self.lens, dtype=torch.int32, device=DEV), PAGE

    def offsets(self, counts):
        return torch.tensor(np.r_[0, np.cumsum(counts)], dtype=torch.int32, device=DEV)

    def attend(self, q, counts):
        heads, table, lens, page = self.call_args()
        kw = dict(cu_q=self.offsets(counts))
        out, lse = nv.nvfp4_kv_attention(q, *self.caches, heads, table, lens, page, max_q=max(counts), return_lse=True, **kw)
        torch.cuda.synchronize()
        assert_attention(out, lse, attention(q, *self.caches, heads, table, lens, page, **kw), "attention")
        return lse

    def weigh(self, q, lse, counts):
        heads, table, lens, page = self.call_args()
        before = self.weights.clone()
        nv.nvfp4_kv_weights(q, lse, self.caches[0], heads, table, lens, page, self.weights, weights=self.weights,
                            cu_q=self.offsets(counts), max_q=max(counts))
        torch.cuda.synchronize()
        ref = received(q, lse, self.caches[0], heads, table, lens, page, before, cu_q=self.offsets(counts))
        assert torch.isfinite(ref[0][ref[2]]).all()
        agree(torch.nan_to_num(self.weights, 7.0), ref, torch.nan_to_num(before, 7.0), "weights")

    def tree(self, m):
        """A tree of m drafts a sequence: attention checked; the accepted path's queries and log-sum-exps."""
        parents = [[-1] + [int(self.r.integers(-1, i)) for i in range(1, m)] for _ in range(self.seqs)]
        bits, depth = np.zeros((self.seqs * m, m), dtype=bool), np.zeros((self.seqs, m), dtype=int)
        for b in range(self.seqs):
            for i, p in enumerate(parents[b]):
                if p >= 0:
                    bits[b * m + i] = bits[b * m + p]
                    depth[b, i] = depth[b, p] + 1
                bits[b * m + i, i] = True
        q = self.append([range(n, n + m) for n in self.lens], [[e + d for d in row] for e, row in zip(self.ends, depth)])
        base = list(self.lens)
        self.lens = [n + m for n in base]
        heads, table, lens, page = self.call_args()
        cu, mask = self.offsets([m] * self.seqs), mask_of(bits).to(DEV)
        out, lse = nv.nvfp4_kv_attention_tree(q, *self.caches, heads, table, lens, page, cu, mask, max_q=m, return_lse=True)
        torch.cuda.synchronize()
        assert_attention(out, lse, tree_attention(q, *self.caches, heads, table, lens, page, cu, mask), "tree")
        # accept the path to some draft (of the last sequence: none)
        paths = [np.flatnonzero(bits[b * m + int(self.r.integers(0, m))]).tolist() for b in range(self.seqs)]
        paths[-1] = []
        moves = np.full((self.seqs, 1, m, 2), -1, dtype=np.int32)
        for b, path in enumerate(paths):
            moves[b, 0, :len(path), 0] = [base[b] + i for i in path]
            moves[b, 0, :len(path), 1] = base[b] + np.arange(len(path))
            for h in range(KVH):
                kept = [self.held[b][h][base[b] + i] for i in path]
                self.held[b][h] = self.held[b][h][:base[b]] + kept
        nv.nvfp4_kv_move(*self.caches, heads, table, page, torch.from_numpy(moves).to(DEV), positions=self.positions)
        self.lens = [n + len(p) for n, p in zip(base, paths)]
        self.ends = [e + len(p) for e, p in zip(self.ends, paths)]
        rows = torch.tensor([b * m + i for b, path in enumerate(paths) for i in path], dtype=torch.long, device=DEV)
        return q[rows].contiguous(), lse[rows].contiguous(), [len(p) for p in paths]

    def evict(self, keep, sinks, recent):
        heads, table, lens, page = self.call_args()
        ends = torch.tensor(self.ends, dtype=torch.int32, device=DEV)
        moves, new = nv.nvfp4_kv_select(self.weights, table, lens, page, keep, positions=self.positions,
                                        next_positions=ends, sinks=sinks, recent=recent)
        torch.cuda.synchronize()
        want, want_lens = chosen(torch.nan_to_num(self.weights, 0.0), self.positions, table, lens, page, keep, ends, sinks,
                                 recent, moves.shape[2])
        np.testing.assert_array_equal(moves.cpu().numpy(), want)
        nv.nvfp4_kv_move(*self.caches, heads, table, page, moves, weights=self.weights, positions=self.positions)
        for b in range(self.seqs):
            for h in range(KVH):
                for src, dst in want[b, h].tolist():
                    if src >= 0:
                        self.held[b][h][dst] = self.held[b][h][src]
                self.held[b][h] = self.held[b][h][:int(want_lens[b])]
        self.lens = new.tolist()
        assert self.lens == want_lens.tolist()

    def check(self, sinks, recent):
        assert nv.nvfp4_get_error() == 0
        for b in range(self.seqs):
            slots = self.slots(b, range(self.lens[b]))
            for h in range(KVH):
                assert len(self.held[b][h]) == self.lens[b]
                pos = self.positions[h].cpu()[slots].tolist()
                assert pos == [x for x, _ in self.held[b][h]]
                for p, (_, want) in enumerate(self.held[b][h]):
                    assert self.row(b, h, p) == want, (b, h, p)
                end = self.ends[b]
                first = [x for x in range(end) if x < sinks or x >= end - recent]
                assert set(first) <= set(pos)  # the first and the most recent ones are still there


@pytest.mark.parametrize("D,keep", [(64, 40), (128, 33)])
def test_drafts_and_a_budget(D, keep):
    layer = Layer(3, 6, D, seed=D)
    prompts = [50, 7, 44]
    step("prompts")
    q = layer.append([range(n) for n in prompts], [range(n) for n in prompts])
    layer.lens, layer.ends = list(prompts), list(prompts)
    layer.weigh(q, layer.attend(q, prompts), prompts)
    layer.evict(keep, 3, 8)
    layer.check(3, 8)
    for i in range(6):
        step(f"tree {i}")
        q, lse, counts = layer.tree([5, 12, 33, 3, 9, 7][i])
        layer.weigh(q, lse, counts)
        layer.evict(keep, 3, 8)
        layer.check(3, 8)
        # the cache as it is now serves single tokens too
        q = layer.append([[n] for n in layer.lens], [[e] for e in layer.ends])
        layer.lens, layer.ends = [n + 1 for n in layer.lens], [e + 1 for e in layer.ends]
        layer.weigh(q, layer.attend(q, [1, 1, 1]), [1, 1, 1])
    layer.evict(keep, 3, 8)
    layer.check(3, 8)
