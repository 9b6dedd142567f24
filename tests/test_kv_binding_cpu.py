"""What the binding of the cache and norm operators refuses before the library sees an address (no GPU
here: tensors that say they are on a device, and a library that notes its calls)."""
import contextlib

import pytest
import torch

import precision_moe_gemm_amd as nv

D, HEADS, N = 64, 2, 3


class OnDevice(torch.Tensor):
    """A tensor that says it is on cuda:0."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))


def dev(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def cache(**parts):
    t = dict(packed=dev(1, 32, D // 2, dtype=torch.uint8), scales=dev(1, 32, D // 16, dtype=torch.uint8),
             global_=dev(1, dtype=torch.float32))
    return nv.NVFP4Tensor(**dict(t, **parts), rows=32, cols=D)


@pytest.fixture
def calls(monkeypatch):
    """The names of the library's calls; none of them is made."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append(name) or 0

    monkeypatch.setattr(nv._lib, "load", Library)
    monkeypatch.setattr(nv, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(nv, "_stream", lambda device=None: 0)
    return made


def append(**kw):
    a = dict(q=None, k=dev(N, HEADS, D), v=dev(N, HEADS, D), slots=dev(N, dtype=torch.int64), k_cache=cache(),
             v_cache=cache())
    return nv.nvfp4_kv_append(**dict(a, **kw))


def attend(**kw):
    a = dict(q=dev(N, 4, D), k_cache=cache(), v_cache=cache(), heads=HEADS, block_table=dev(N, 1, dtype=torch.int32),
             kv_lens=dev(N, dtype=torch.int32), page_size=16, out=dev(N, 4, D), ws=dev(1 << 10, dtype=torch.uint8))
    return nv.nvfp4_kv_attention(**dict(a, **kw))


def test_the_calls_as_they_stand_reach_the_library(calls):
    append()
    attend()
    assert calls == ["nvfp4_kv_append", "nvfp4_kv_attention"]


ELSEWHERE = [dict(packed=torch.zeros((1, 32, D // 2), dtype=torch.uint8)),
             dict(scales=torch.zeros((1, 32, D // 16), dtype=torch.uint8)), dict(global_=torch.zeros(1))]


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("which", ["k_cache", "v_cache"])
@pytest.mark.parametrize("parts", ELSEWHERE, ids=["packed", "scales", "global"])
def test_a_cache_that_lies_elsewhere(calls, call, which, parts):
    """Any part of either cache on the host: its address must not reach a kernel."""
    with pytest.raises(ValueError):
        call(**{which: cache(**parts)})
    assert calls == []


@pytest.mark.parametrize("name", ["heads", "page_size", "max_q", "window"])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 16, -(1 << 32) + 16])
def test_numbers_past_32_bits(calls, name, value):
    """The C types would take them modulo 2^32: a window of 2^32 + 16 as one of 16."""
    with pytest.raises(ValueError):
        attend(**{name: value})
    assert calls == []


def test_heads_that_contradict_the_operands(calls):
    for kw in (dict(heads=4), dict(heads=1, k=None), dict(heads=3, v=None)):
        with pytest.raises(ValueError):
            append(**kw)
    with pytest.raises(ValueError):
        append(q=dev(N, 4, D), k=None, v=None, heads=(1 << 32) + 2)
    assert calls == []
    append(heads=2)
    append(heads=2, v=None)
    assert calls == ["nvfp4_kv_append"] * 2
