"""Refusals of nvfp4_kv_append, nvfp4_kv_attention and mxfp8_add_rmsnorm: found on the host, before any
launch (no GPU here), and the same under the sanitizer build of the host layer."""
import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from precision_moe_gemm_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


def cache(rows=64, cols=128, batch=1, flags=0, packed=4096, scales=8192, glob=64):
    from precision_moe_gemm_amd import _lib
    return _lib.NVFP4TensorC(packed, scales, glob, rows, cols, batch, flags)


APPEND = dict(q=P(4096), ld_q=512, q_heads=4, k=P(8192), ld_k=256, v=P(12288), ld_v=256, heads=2, n=3, slots=P(64),
              pos=P(64), cs=P(64), max_pos=10, rot=128, inter=0, q_out=P(16384), ld_qo=512, kc=None, vc=None)


def append(lib, **kw):
    a = dict(APPEND, **kw)
    kc, vc = a["kc"] or cache(), a["vc"] or cache()
    return lib.nvfp4_kv_append(a["q"], a["ld_q"], a["q_heads"], a["k"], a["ld_k"], a["v"], a["ld_v"], a["heads"],
                               a["n"], a["slots"], a["pos"], a["cs"], a["max_pos"], a["rot"], a["inter"], a["q_out"],
                               a["ld_qo"], ctypes.byref(kc), ctypes.byref(vc), None)


def test_append_refusals(lib):
    from precision_moe_gemm_amd import _lib as L
    assert append(lib, n=0) == L.OK
    assert append(lib, q=None, k=None, v=None) == L.OK
    assert append(lib, n=-1) == L.SHAPE
    assert append(lib, heads=0) == L.SHAPE
    assert append(lib, heads=3) == L.SHAPE                      # 64 rows are no whole tokens of 3 heads
    assert append(lib, q_heads=0) == L.SHAPE
    assert append(lib, ld_q=504) == L.SHAPE
    assert append(lib, ld_k=252) == L.SHAPE
    assert append(lib, ld_v=260) == L.SHAPE                     # not a multiple of 8
    assert append(lib, ld_qo=8) == L.SHAPE
    assert append(lib, rot=160) == L.SHAPE
    assert append(lib, rot=-32) == L.SHAPE
    assert append(lib, rot=48) == L.UNSUPPORTED
    assert append(lib, max_pos=0) == L.SHAPE
    assert append(lib, vc=cache(cols=64)) == L.SHAPE
    assert append(lib, vc=cache(rows=128)) == L.SHAPE
    assert append(lib, kc=cache(batch=2)) == L.SHAPE
    assert append(lib, kc=cache(cols=144), vc=cache(cols=144), ld_q=1024, ld_k=512, ld_v=512, ld_qo=1024) == L.UNSUPPORTED
    assert append(lib, kc=cache(glob=0)) == L.INVALID_ARG
    assert append(lib, kc=cache(packed=4097)) == L.INVALID_ARG
    assert append(lib, kc=cache(flags=L.TILED_SCALES)) == L.UNSUPPORTED
    for name in ("q", "k", "v", "q_out"):
        assert append(lib, **{name: P(4098)}) == L.INVALID_ARG, name
    assert append(lib, q_out=None) == L.INVALID_ARG
    assert append(lib, slots=None) == L.INVALID_ARG
    assert append(lib, slots=P(4)) == L.INVALID_ARG
    assert append(lib, pos=None) == L.INVALID_ARG
    assert append(lib, cs=None) == L.INVALID_ARG
    assert append(lib, cs=P(72)) == L.INVALID_ARG


ATTEND = dict(q=P(4096), ld_q=512, n=3, q_heads=4, kc=None, vc=None, heads=2, table=P(64), ld_table=2, pages=2, page=16,
              lens=P(64), cu=None, seqs=3, max_q=1, scale=0.1, causal=1, window=0, out=P(8192), ld_out=512, lse=None,
              ws=None, ws_bytes=None)


def attend(lib, **kw):
    from precision_moe_gemm_amd import _lib as L
    a = dict(ATTEND, **kw)
    kc, vc = a["kc"] or cache(), a["vc"] or cache()
    need = lib.nvfp4_workspace_size(L.OP_KV_ATTENTION, max(a["n"], 0), max(a["q_heads"], 0), a["heads"], kc.cols,
                                    max(a["seqs"], 0))
    ws = a["ws"] or P(1 << 20)
    return lib.nvfp4_kv_attention(a["q"], a["ld_q"], a["n"], a["q_heads"], ctypes.byref(kc), ctypes.byref(vc),
                                  a["heads"], a["table"], a["ld_table"], a["pages"], a["page"], a["lens"], a["cu"],
                                  a["seqs"], a["max_q"], a["scale"], a["causal"], a["window"], a["out"], a["ld_out"],
                                  a["lse"], ws, need if a["ws_bytes"] is None else a["ws_bytes"], None)


def test_attention_refusals(lib):
    from precision_moe_gemm_amd import _lib as L
    assert attend(lib, n=0, seqs=0) == L.OK
    assert attend(lib, seqs=0, cu=P(64)) == L.OK
    assert attend(lib, n=-1) == L.SHAPE
    assert attend(lib, seqs=-1) == L.SHAPE
    assert attend(lib, seqs=2) == L.SHAPE                       # without cu_q: one row per sequence
    assert attend(lib, q_heads=5) == L.SHAPE
    assert attend(lib, heads=0) == L.SHAPE
    assert attend(lib, heads=3, q_heads=3) == L.SHAPE           # 64 rows are no whole tokens of 3 heads
    assert attend(lib, pages=-1) == L.SHAPE
    assert attend(lib, ld_table=1) == L.SHAPE
    assert attend(lib, page=0) == L.SHAPE
    assert attend(lib, page=64) == L.SHAPE                      # 32 tokens hold no page of 64
    assert attend(lib, page=24) == L.UNSUPPORTED
    assert attend(lib, max_q=-1) == L.SHAPE
    assert attend(lib, ld_q=504) == L.SHAPE
    assert attend(lib, ld_out=516) == L.SHAPE
    assert attend(lib, vc=cache(cols=64)) == L.SHAPE
    assert attend(lib, vc=cache(rows=128)) == L.SHAPE
    assert attend(lib, kc=cache(batch=3)) == L.SHAPE
    assert attend(lib, kc=cache(cols=96), vc=cache(cols=96)) == L.UNSUPPORTED
    assert attend(lib, pages=1 << 30, ld_table=1 << 30) == L.UNSUPPORTED
    assert attend(lib, kc=cache(glob=0)) == L.INVALID_ARG
    assert attend(lib, kc=cache(flags=L.TILED_SCALES)) == L.UNSUPPORTED
    for v in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(lib, scale=v) == L.INVALID_ARG, v
    assert attend(lib, window=-1) == L.INVALID_ARG
    assert attend(lib, causal=0, window=5) == L.INVALID_ARG
    for name in ("q", "out", "lens", "table"):
        assert attend(lib, **{name: None}) == L.INVALID_ARG, name
    assert attend(lib, q=P(4098)) == L.INVALID_ARG
    assert attend(lib, out=P(8200)) == L.INVALID_ARG
    assert attend(lib, lens=P(66)) == L.INVALID_ARG
    assert attend(lib, lse=P(66)) == L.INVALID_ARG
    assert attend(lib, cu=P(66)) == L.INVALID_ARG


def test_attention_workspace_and_limits(lib):
    from precision_moe_gemm_amd import _lib as L
    need = lib.nvfp4_workspace_size(L.OP_KV_ATTENTION, 3, 4, 2, 128, 3)
    assert need > 0 and need % 256 == 0
    assert attend(lib, ws_bytes=need - 1) == L.WORKSPACE
    assert attend(lib, ws_bytes=0) == L.WORKSPACE
    assert attend(lib, ws=P((1 << 20) + 128)) == L.INVALID_ARG
    c = cache()
    a = dict(ATTEND)
    args = [a["q"], a["ld_q"], 3, 4, ctypes.byref(c), ctypes.byref(c), 2, a["table"], 2, 2, 16, a["lens"], None, 3, 1,
            0.1, 1, 0, a["out"], a["ld_out"], None, None, need, None]
    assert lib.nvfp4_kv_attention(*args) == L.INVALID_ARG       # no workspace
    for n in (0, -1):
        assert lib.nvfp4_workspace_size(L.OP_KV_ATTENTION, n, 4, 2, 128, 3) == 0
        assert lib.nvfp4_workspace_size(L.OP_KV_ATTENTION, 3, 4, 2, 128, n) == 0
    huge = cache(rows=2 << 31)
    assert attend(lib, kc=huge, vc=huge) == L.UNSUPPORTED       # 2^31 tokens of 2 heads
    many = cache(rows=65536 * 16, cols=64)
    assert attend(lib, kc=many, vc=many, heads=65536, q_heads=65536, ld_q=1 << 22, ld_out=1 << 22, pages=1,
                  ld_table=1, page=16) == L.UNSUPPORTED
    assert attend(lib, n=1 << 30, seqs=1 << 30) == L.UNSUPPORTED  # 2^32 rows of queries


def test_device_tensors_only(lib):
    """A tensor of the host is refused before anything is launched on its address."""
    import torch

    import precision_moe_gemm_amd as nv
    t = nv.NVFP4Tensor.empty(4, 64, 1, "cpu")
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        nv.nvfp4_audit_scales(t)
    with pytest.raises(ValueError):
        nv._stream("cpu")
    with pytest.raises(ValueError):
        nv._stream(torch.device("cpu"))


NORM = dict(x=P(4096), ld_x=64, res=P(8192), ld_res=64, w=P(64), eps=1e-6, rows=3, cols=64, sum=P(12288), ld_sum=64,
            y=P(16384), ld_y=64, fp8=P(20480), e8=P(24576))


def norm(lib, **kw):
    a = dict(NORM, **kw)
    return lib.mxfp8_add_rmsnorm(a["x"], a["ld_x"], a["res"], a["ld_res"], a["w"], a["eps"], a["rows"], a["cols"],
                                 a["sum"], a["ld_sum"], a["y"], a["ld_y"], a["fp8"], a["e8"], None)


def test_norm_refusals(lib):
    from precision_moe_gemm_amd import _lib as L
    assert norm(lib, rows=0) == L.OK
    assert norm(lib, rows=-1) == L.SHAPE
    assert norm(lib, cols=48) == L.SHAPE
    for name in ("ld_x", "ld_res", "ld_sum", "ld_y"):
        assert norm(lib, **{name: 56}) == L.SHAPE, name
        assert norm(lib, **{name: 68}) == L.SHAPE, name
    for name in ("x", "res", "w", "sum", "y", "fp8"):
        assert norm(lib, **{name: P(4100)}) == L.INVALID_ARG, name
    assert norm(lib, x=None) == L.INVALID_ARG
    assert norm(lib, fp8=None) == L.INVALID_ARG
    assert norm(lib, e8=None) == L.INVALID_ARG
    for v in (-1e-6, float("nan"), float("inf")):
        assert norm(lib, eps=v) == L.INVALID_ARG, v
    wide = dict(cols=65536 + 32, ld_x=70000, ld_res=70000, ld_sum=70000, ld_y=70000)
    assert norm(lib, **wide) == L.UNSUPPORTED


@pytest.mark.skipif("NVFP4_LIB_PATH" in os.environ, reason="this run is the sanitized one")
def test_refusals_under_asan_ubsan():
    from precision_moe_gemm_amd import build
    env = dict(os.environ, LD_PRELOAD=build.sanitizer_runtime(), NVFP4_LIB_PATH=build.build_sanitized(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_abi_kv_cpu.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
