"""What the binding of the operators for trees and for caches of bounded length refuses before the library sees
an address (no GPU here: tensors that say they are on a device, and a library that notes its calls)."""
import pytest
import torch

import precision_moe_gemm_amd as nv
from tests.test_kv_binding_cpu import D, HEADS, N, cache, calls, dev  # noqa: F401  (calls: the fixture)

TOKENS = 32 // HEADS


def i32(*shape):
    return dev(*shape, dtype=torch.int32)


def f32(*shape):
    return dev(*shape, dtype=torch.float32)


def tree(**kw):
    a = dict(q=dev(N, 4, D), k_cache=cache(), v_cache=cache(), heads=HEADS, block_table=i32(N, 1), kv_lens=i32(N),
             page_size=16, cu_q=i32(N + 1), mask=i32(N, 1), out=dev(N, 4, D), ws=dev(1 << 10, dtype=torch.uint8))
    return nv.nvfp4_kv_attention_tree(**dict(a, **kw))


def weights(**kw):
    a = dict(q=dev(N, 4, D), lse=f32(N, 4), k_cache=cache(), heads=HEADS, block_table=i32(N, 1), kv_lens=i32(N),
             page_size=16, out=f32(HEADS, TOKENS), weights=f32(HEADS, TOKENS), ws=dev(1 << 10, dtype=torch.uint8))
    return nv.nvfp4_kv_weights(**dict(a, **kw))


def move(**kw):
    a = dict(k_cache=cache(), v_cache=cache(), heads=HEADS, block_table=i32(N, 1), page_size=16, moves=i32(N, HEADS, 2, 2),
             weights=f32(HEADS, TOKENS), positions=i32(HEADS, TOKENS))
    return nv.nvfp4_kv_move(**dict(a, **kw))


def test_the_calls_as_they_stand_reach_the_library(calls):
    tree()
    weights()
    weights(weights=None)
    move()
    move(weights=None, positions=None, moves=i32(N, 1, 5, 2))
    assert calls == ["nvfp4_kv_attention_tree"] + 2 * ["nvfp4_kv_weights"] + 2 * ["nvfp4_kv_move"]


ELSEWHERE = [dict(packed=torch.zeros((1, 32, D // 2), dtype=torch.uint8)),
             dict(scales=torch.zeros((1, 32, D // 16), dtype=torch.uint8)), dict(global_=torch.zeros(1))]


@pytest.mark.parametrize("call,which", [(tree, "k_cache"), (tree, "v_cache"), (weights, "k_cache"), (move, "k_cache"),
                                        (move, "v_cache")])
@pytest.mark.parametrize("parts", ELSEWHERE, ids=["packed", "scales", "global"])
def test_a_cache_that_lies_elsewhere(calls, call, which, parts):
    with pytest.raises(ValueError):
        call(**{which: cache(**parts)})
    assert calls == []


@pytest.mark.parametrize("call,name", [(tree, "mask"), (tree, "cu_q"), (tree, "block_table"), (weights, "lse"),
                                       (weights, "out"), (weights, "weights"), (weights, "kv_lens"), (move, "moves"),
                                       (move, "weights"), (move, "positions"), (move, "block_table")])
def test_an_operand_that_lies_elsewhere(calls, call, name):
    """On the host: its address must not reach a kernel."""
    shapes = dict(mask=(N, 1), cu_q=(N + 1,), block_table=(N, 1), lse=(N, 4), out=(HEADS, TOKENS),
                  weights=(HEADS, TOKENS), kv_lens=(N,), moves=(N, HEADS, 2, 2), positions=(HEADS, TOKENS))
    dtype = torch.float32 if name in ("lse", "out", "weights") else torch.int32
    with pytest.raises(ValueError):
        call(**{name: torch.zeros(shapes[name], dtype=dtype)})
    assert calls == []


@pytest.mark.parametrize("call,name", [(tree, "heads"), (tree, "page_size"), (tree, "max_q"), (tree, "window"),
                                       (weights, "max_q"), (weights, "page_size"), (weights, "window"),
                                       (move, "page_size")])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 16, -(1 << 32) + 16])
def test_numbers_past_32_bits(calls, call, name, value):
    with pytest.raises(ValueError):
        call(**{name: value})
    assert calls == []


def test_shapes_that_contradict_each_other(calls):
    for kw in (dict(mask=i32(N + 1, 1)), dict(mask=i32(N, 1).expand(N, 2)), dict(mask=f32(N, 1)), dict(cu_q=i32(N)),
               dict(kv_lens=i32(N + 1)), dict(out=dev(N, 4, D + 8))):
        with pytest.raises(ValueError):
            tree(**kw)
    for kw in (dict(lse=f32(N, 3)), dict(lse=f32(4, N).T), dict(out=f32(HEADS, TOKENS + 1)), dict(weights=f32(1, TOKENS)),
               dict(out=f32(1, TOKENS).expand(HEADS, TOKENS)), dict(heads=1), dict(cu_q=i32(N)), dict(q=dev(N, 4, 32))):
        with pytest.raises(ValueError):
            weights(**kw)
    for kw in (dict(moves=i32(N + 1, HEADS, 2, 2)), dict(moves=i32(N, HEADS, 2, 3)), dict(moves=i32(N, HEADS, 2)),
               dict(moves=i32(N, 2, HEADS, 2).transpose(1, 2)[:, :, :1]), dict(weights=f32(HEADS, TOKENS - 1)),
               dict(positions=f32(HEADS, TOKENS)), dict(heads=1)):
        with pytest.raises(ValueError):
            move(**kw)
    assert calls == []
