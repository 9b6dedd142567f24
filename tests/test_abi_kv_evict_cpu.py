"""Refusals of nvfp4_kv_attention_tree, nvfp4_kv_weights, nvfp4_kv_select and nvfp4_kv_move: found on the host,
before any launch (no GPU here), and the same under the sanitizer build of the host layer."""
import ctypes
import os
import subprocess
import sys

import pytest

from tests.test_abi_kv_cpu import ATTEND, P, ROOT, cache, lib  # noqa: F401  (lib: the fixture)

TREE = dict({k: v for k, v in ATTEND.items() if k != "causal"}, mask=P(64), ld_mask=1, words=1)


def tree(lib, **kw):
    from precision_moe_gemm_amd import _lib as L
    a = dict(TREE, **kw)
    kc, vc = a["kc"] or cache(), a["vc"] or cache()
    need = lib.nvfp4_workspace_size(L.OP_KV_ATTENTION_TREE, max(a["n"], 0), max(a["q_heads"], 0), a["heads"], kc.cols,
                                    max(a["seqs"], 0))
    return lib.nvfp4_kv_attention_tree(a["q"], a["ld_q"], a["n"], a["q_heads"], ctypes.byref(kc), ctypes.byref(vc),
                                       a["heads"], a["table"], a["ld_table"], a["pages"], a["page"], a["lens"], a["cu"],
                                       a["seqs"], a["max_q"], a["mask"], a["ld_mask"], a["words"], a["scale"],
                                       a["window"], a["out"], a["ld_out"], a["lse"], a["ws"] or P(1 << 20),
                                       need if a["ws_bytes"] is None else a["ws_bytes"], None)


def test_tree_refusals(lib):
    from precision_moe_gemm_amd import _lib as L
    short = dict(ws_bytes=0)  # (stops what is not refused before a launch)
    assert tree(lib, **short) == L.WORKSPACE
    assert tree(lib, n=0, seqs=0) == L.OK
    assert tree(lib, n=-1) == L.SHAPE
    assert tree(lib, seqs=2) == L.SHAPE
    assert tree(lib, q_heads=5) == L.SHAPE
    assert tree(lib, words=-1, ld_mask=0) == L.SHAPE
    assert tree(lib, words=2) == L.SHAPE                        # a row stride below the words
    assert tree(lib, mask=None) == L.INVALID_ARG
    assert tree(lib, mask=P(66)) == L.INVALID_ARG
    assert tree(lib, mask=None, words=0, **short) == L.WORKSPACE
    assert tree(lib, ld_mask=7, **short) == L.WORKSPACE
    assert tree(lib, page=24) == L.UNSUPPORTED
    assert tree(lib, window=-1) == L.INVALID_ARG
    assert tree(lib, window=5, **short) == L.WORKSPACE
    for v in (0.0, -1.0, float("nan"), float("inf")):
        assert tree(lib, scale=v) == L.INVALID_ARG, v
    assert tree(lib, out=P(4096 + 16)) == L.INVALID_ARG         # shares memory with q
    assert tree(lib, kc=cache(cols=96), vc=cache(cols=96)) == L.UNSUPPORTED
    for name in ("q", "out", "lens", "table"):
        assert tree(lib, **{name: None}) == L.INVALID_ARG, name


def test_tree_workspace(lib):
    """Two slots of the tile kernel's 256 workgroups for heads of 256: their 128 rows of 260 numbers (the row
    kernel's slots take 264, the list of tiles a few KB)."""
    from precision_moe_gemm_amd import _lib as L
    for heads in (1, 4, 8):
        need = lib.nvfp4_workspace_size(L.OP_KV_ATTENTION_TREE, 64, 8 * heads, heads, 256, 1)
        slots = 256 * 2 * 128 * 260 * 4
        assert slots <= need < slots * 1.02, heads


WEIGHTS = dict(q=P(4096), ld_q=512, n=3, q_heads=4, lse=P(64), kc=None, heads=2, table=P(64), ld_table=2, pages=2, page=16,
               lens=P(64), cu=None, seqs=3, max_q=1, scale=0.1, causal=1, window=0, w=P(1 << 14), ld_w=32, out=P(1 << 15),
               ld_out=32, ws=P(1 << 20), ws_bytes=None)


def weights(lib, **kw):
    from precision_moe_gemm_amd import _lib as L
    a = dict(WEIGHTS, **kw)
    kc = a["kc"] or cache()
    need = lib.nvfp4_workspace_size(L.OP_KV_WEIGHTS, max(a["n"], 0), max(a["q_heads"], 0), a["heads"], kc.cols,
                                    max(a["seqs"], 0))
    return lib.nvfp4_kv_weights(a["q"], a["ld_q"], a["n"], a["q_heads"], a["lse"], ctypes.byref(kc), a["heads"],
                                a["table"], a["ld_table"], a["pages"], a["page"], a["lens"], a["cu"], a["seqs"],
                                a["max_q"], a["scale"], a["causal"], a["window"], a["w"], a["ld_w"], a["out"],
                                a["ld_out"], a["ws"], need if a["ws_bytes"] is None else a["ws_bytes"], None)


def test_weights_refusals(lib):
    from precision_moe_gemm_amd import _lib as L
    short = dict(ws_bytes=0)
    assert weights(lib, **short) == L.WORKSPACE
    assert weights(lib, n=0, seqs=0) == L.OK
    assert weights(lib, pages=0, ld_table=0, table=None) == L.OK  # no cached token
    assert weights(lib, n=-1) == L.SHAPE
    assert weights(lib, seqs=-1, cu=P(64)) == L.SHAPE
    assert weights(lib, seqs=2) == L.SHAPE
    assert weights(lib, q_heads=5) == L.SHAPE
    assert weights(lib, heads=0) == L.SHAPE
    assert weights(lib, heads=3, q_heads=3) == L.SHAPE
    assert weights(lib, pages=-1) == L.SHAPE
    assert weights(lib, ld_table=1) == L.SHAPE
    assert weights(lib, page=0) == L.SHAPE
    assert weights(lib, page=64) == L.SHAPE
    assert weights(lib, page=24) == L.UNSUPPORTED
    assert weights(lib, max_q=-1) == L.SHAPE
    assert weights(lib, ld_q=504) == L.SHAPE
    assert weights(lib, ld_q=516) == L.SHAPE
    assert weights(lib, ld_w=31) == L.SHAPE
    assert weights(lib, ld_out=31) == L.SHAPE
    assert weights(lib, w=None, ld_w=0, **short) == L.WORKSPACE
    assert weights(lib, kc=cache(batch=2)) == L.SHAPE
    assert weights(lib, kc=cache(cols=96)) == L.UNSUPPORTED
    assert weights(lib, kc=cache(glob=0)) == L.INVALID_ARG
    assert weights(lib, kc=cache(flags=L.TILED_SCALES)) == L.UNSUPPORTED
    assert weights(lib, pages=1 << 27, ld_table=1 << 27) == L.UNSUPPORTED
    assert weights(lib, n=1 << 30, seqs=1 << 30) == L.UNSUPPORTED
    for v in (0.0, -1.0, float("nan"), float("inf")):
        assert weights(lib, scale=v) == L.INVALID_ARG, v
    assert weights(lib, window=-1) == L.INVALID_ARG
    assert weights(lib, causal=0, window=5) == L.INVALID_ARG
    for name in ("q", "lse", "lens", "table", "out"):
        assert weights(lib, **{name: None}) == L.INVALID_ARG, name
        assert weights(lib, **{name: P(WEIGHTS[name].value + 2)}) == L.INVALID_ARG, name
    assert weights(lib, w=P((1 << 14) + 2)) == L.INVALID_ARG
    assert weights(lib, cu=P(66)) == L.INVALID_ARG
    assert weights(lib, ws=None) == L.INVALID_ARG
    assert weights(lib, ws=P((1 << 20) + 128)) == L.INVALID_ARG
    wide = cache(cols=256, scales=8196)
    assert weights(lib, kc=wide, ld_q=1024) == L.INVALID_ARG     # 16-byte copies of scales


def test_weights_without_query_rows(lib):
    """They are copied, by launches that need the workspace as well."""
    from precision_moe_gemm_amd import _lib as L
    assert lib.nvfp4_workspace_size(L.OP_KV_WEIGHTS, 0, 4, 2, 128, 3) == lib.nvfp4_workspace_size(L.OP_KV_WEIGHTS, 3, 4, 2, 128, 3)
    assert weights(lib, n=0, cu=P(64), q=None, lse=None, ws=None) == L.INVALID_ARG
    assert weights(lib, n=0, cu=P(64), q=None, lse=None, ws_bytes=0) == L.WORKSPACE


def test_weights_in_place_or_elsewhere(lib):
    """Two rows of 32 numbers: in place with the same stride alone, side by side in one buffer."""
    from precision_moe_gemm_amd import _lib as L
    at = 1 << 16

    def refused(out, ld_w=32, ld_out=32):
        s = weights(lib, w=P(at), out=P(out), ld_w=ld_w, ld_out=ld_out, ws_bytes=0)
        assert s in (L.INVALID_ARG, L.WORKSPACE)
        return s == L.INVALID_ARG

    assert not refused(at)
    assert refused(at, 32, 40)
    assert refused(at + 4) and refused(at + 252) and refused(at - 252)
    assert not refused(at + 256) and not refused(at - 256)
    assert not refused(at + 128, 64, 64)
    assert refused(at + 124, 64, 64)


SELECT = dict(w=P(1 << 14), ld_w=64, pos=P(1 << 15), ld_p=64, heads=2, tokens=64, table=P(64), ld_table=3, pages=3, page=16,
              lens=P(64), next=P(64), seqs=3, keep=20, sinks=2, recent=8, moves=P(4096), cap=20, out=P(8192), ws=None, ws_bytes=0)


def select(lib, **kw):
    a = dict(SELECT, **kw)
    return lib.nvfp4_kv_select(a["w"], a["ld_w"], a["pos"], a["ld_p"], a["heads"], a["tokens"], a["table"], a["ld_table"],
                               a["pages"], a["page"], a["lens"], a["next"], a["seqs"], a["keep"], a["sinks"], a["recent"],
                               a["moves"], a["cap"], a["out"], a["ws"], a["ws_bytes"], None)


def test_select_refusals(lib):
    from precision_moe_gemm_amd import _lib as L
    assert select(lib, seqs=0) == L.OK
    assert select(lib, seqs=-1) == L.SHAPE
    assert select(lib, heads=0) == L.SHAPE
    assert select(lib, tokens=-1) == L.SHAPE
    assert select(lib, tokens=15, ld_w=64) == L.SHAPE           # no page
    assert select(lib, pages=-1) == L.SHAPE
    assert select(lib, ld_table=2) == L.SHAPE
    assert select(lib, page=0) == L.SHAPE
    assert select(lib, page=24) == L.UNSUPPORTED
    assert select(lib, tokens=1 << 31, ld_w=1 << 31, ld_p=1 << 31) == L.UNSUPPORTED
    assert select(lib, pages=1 << 27, ld_table=1 << 27) == L.UNSUPPORTED
    assert select(lib, heads=70000) == L.UNSUPPORTED
    assert select(lib, seqs=1 << 22) == L.UNSUPPORTED
    assert select(lib, ld_w=63) == L.SHAPE
    assert select(lib, ld_p=63) == L.SHAPE
    assert select(lib, cap=19) == L.SHAPE                       # min(20, 48 - 20) moves are possible
    assert select(lib, keep=40, cap=7) == L.SHAPE               # 48 - 40
    assert select(lib, cap=-1, keep=48) == L.SHAPE
    for name, v in (("keep", 0), ("keep", -1), ("sinks", -1), ("recent", -1), ("recent", 19)):
        assert select(lib, **{name: v}) == L.INVALID_ARG, (name, v)
    for name in ("w", "lens", "table", "moves", "out", "next"):
        assert select(lib, **{name: None}) == L.INVALID_ARG, name
        assert select(lib, **{name: P(SELECT[name].value + 2)}) == L.INVALID_ARG, name
    assert select(lib, pos=P(66)) == L.INVALID_ARG
    assert select(lib, out=SELECT["lens"]) == L.INVALID_ARG     # other heads still read the lengths
    assert select(lib, out=P(256), next=P(256)) == L.INVALID_ARG
    assert select(lib, cap=1 << 30) == L.UNSUPPORTED
    assert select(lib, out=P(64 + 8)) == L.INVALID_ARG


def test_select_workspace(lib):
    from precision_moe_gemm_amd import _lib as L
    assert lib.nvfp4_workspace_size(L.OP_KV_SELECT, 0, 0, 2, 32768, 3) == 0
    need = lib.nvfp4_workspace_size(L.OP_KV_SELECT, 0, 0, 2, 32784, 3)
    assert need >= 2 * 32784 * 3 * 4 and need % 256 == 0
    assert lib.nvfp4_workspace_size(L.OP_KV_SELECT, 0, 0, 0, 32784, 3) == 0
    assert lib.nvfp4_workspace_size(L.OP_KV_SELECT, 0, 0, 2, 32784, -1) == 0
    wide = dict(tokens=1 << 20, ld_w=1 << 20, ld_p=1 << 20, pages=2049, ld_table=2049, keep=16, sinks=0)
    assert select(lib, **wide) == L.INVALID_ARG                 # no workspace
    assert select(lib, ws=P((1 << 20) + 128), ws_bytes=need, **wide) == L.INVALID_ARG
    assert select(lib, ws=P(1 << 20), ws_bytes=need - 1, **wide) == L.WORKSPACE


MOVE = dict(kc=None, vc=None, heads=2, table=P(64), ld_table=2, pages=2, page=16, seqs=3, moves=P(4096), lists=2, cap=5,
            w=P(1 << 14), ld_w=32, pos=P(1 << 15), ld_p=32)


def move(lib, **kw):
    a = dict(MOVE, **kw)
    kc, vc = a["kc"] or cache(), a["vc"] or cache()
    return lib.nvfp4_kv_move(ctypes.byref(kc), ctypes.byref(vc), a["heads"], a["table"], a["ld_table"], a["pages"],
                             a["page"], a["seqs"], a["moves"], a["lists"], a["cap"], a["w"], a["ld_w"], a["pos"],
                             a["ld_p"], None)


def test_move_refusals(lib):
    from precision_moe_gemm_amd import _lib as L
    assert move(lib, seqs=0) == L.OK
    assert move(lib, cap=0) == L.OK
    assert move(lib, pages=0, ld_table=0, table=None) == L.OK
    assert move(lib, seqs=-1) == L.SHAPE
    assert move(lib, heads=0, lists=1) == L.SHAPE
    assert move(lib, heads=3, lists=3) == L.SHAPE
    assert move(lib, lists=3) == L.SHAPE
    assert move(lib, lists=0) == L.SHAPE
    assert move(lib, cap=-1) == L.SHAPE
    assert move(lib, ld_table=1) == L.SHAPE
    assert move(lib, page=64) == L.SHAPE
    assert move(lib, page=24) == L.UNSUPPORTED
    assert move(lib, ld_w=31) == L.SHAPE
    assert move(lib, ld_p=31) == L.SHAPE
    assert move(lib, vc=cache(cols=64)) == L.SHAPE
    assert move(lib, vc=cache(rows=128)) == L.SHAPE
    assert move(lib, kc=cache(batch=3)) == L.SHAPE
    assert move(lib, kc=cache(cols=144), vc=cache(cols=144)) == L.UNSUPPORTED
    assert move(lib, kc=cache(cols=8192), vc=cache(cols=8192)) == L.UNSUPPORTED
    assert move(lib, cap=1 << 30) == L.UNSUPPORTED
    assert move(lib, kc=cache(packed=4104)) == L.INVALID_ARG
    assert move(lib, vc=cache(flags=L.TILED_SCALES)) == L.UNSUPPORTED
    for name in ("table", "moves"):
        assert move(lib, **{name: None}) == L.INVALID_ARG, name
        assert move(lib, **{name: P(MOVE[name].value + 2)}) == L.INVALID_ARG, name
    assert move(lib, w=P(66)) == L.INVALID_ARG
    assert move(lib, pos=P(66)) == L.INVALID_ARG


def test_move_of_caches_that_share_memory(lib):
    """K and V are one tensor, or lie apart: 64 rows of 64 bytes of codes and 8 of scales."""
    from precision_moe_gemm_amd import _lib as L
    k, s = 1 << 20, 1 << 21

    def refused(packed, scales):
        kc, vc = cache(packed=k, scales=s), cache(packed=packed, scales=scales)
        got = move(lib, kc=kc, vc=vc, cap=1 << 30)                  # (stops what is not refused before a launch)
        assert got in (L.INVALID_ARG, L.UNSUPPORTED) and got == move(lib, kc=vc, vc=kc, cap=1 << 30)
        return got == L.INVALID_ARG

    assert not refused(k, s)
    for packed, scales in ((4096, 512), (-4096, -512), (4096, -512), (8192, 4096)):
        assert not refused(k + packed, s + scales), (packed, scales)
    for packed, scales in ((4096, 0), (0, 512), (16, 512), (4080, 512), (-4080, 512), (4096, 4), (4096, 508), (4096, -508),
                           (16, 4)):
        assert refused(k + packed, s + scales), (packed, scales)


@pytest.mark.skipif("NVFP4_LIB_PATH" in os.environ, reason="this run is the sanitized one")
def test_refusals_under_asan_ubsan():
    from precision_moe_gemm_amd import build
    env = dict(os.environ, LD_PRELOAD=build.sanitizer_runtime(), NVFP4_LIB_PATH=build.build_sanitized(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_abi_kv_evict_cpu.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
