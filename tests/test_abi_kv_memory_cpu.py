"""Refusals of the cache and norm operators that concern where their operands lie: found on the host, before
any launch (no GPU here), and the same under the sanitizer build of the host layer."""
import os
import subprocess
import sys

import pytest

from tests.test_abi_kv_cpu import P, ROOT, append, attend, cache, lib, norm  # noqa: F401  (lib: the fixture)


def test_attention_scales_of_256_wide_heads_are_copied_16_bytes_at_a_time(lib):
    """check_tensor asks for 4 bytes; with D = 256 the row kernel copies 16 per lane."""
    from precision_moe_gemm_amd import _lib as L
    wide = dict(ld_q=1024, ld_out=1024, q_heads=4, out=P(1 << 20))
    short = dict(ws_bytes=0)  # (stops what is not refused before a launch)
    good = cache(cols=256)
    assert attend(lib, kc=good, vc=good, **wide, **short) == L.WORKSPACE
    for off in (4, 8, 12):
        bad = cache(cols=256, scales=8192 + off)
        assert attend(lib, kc=bad, vc=good, **wide, **short) == L.INVALID_ARG, off
        assert attend(lib, kc=good, vc=bad, **wide, **short) == L.INVALID_ARG, off
    for cols in (64, 128):  # copies of 4 bytes
        odd = cache(cols=cols, scales=8196)
        assert attend(lib, kc=odd, vc=odd, **short) == L.WORKSPACE, cols


def test_attention_out_must_not_share_memory_with_q(lib):
    """Workgroups write their rows while others still read q: 3 rows of 512 elements, 1024 bytes each."""
    from precision_moe_gemm_amd import _lib as L
    q, end = 1 << 16, 3 * 1024  # (end: behind three dense rows)
    for out, ld_q, ld_out in ((q, 512, 512), (q + 16, 512, 512), (q - 16, 512, 512), (q + 1024, 512, 512),
                              (q + end - 16, 512, 512), (q - end + 16, 512, 512), (q, 1024, 512), (q, 512, 1024),
                              (q + 2048, 1024, 1024),              # out's row 0 is q's row 1
                              (q + 1040, 1024, 1024),              # out's row 0 ends in q's row 1
                              (q - 2064, 1024, 1024),              # q's row 0 begins in out's row 1
                              (q + 1024, 1024, 512), (q - 1024, 512, 1024), (q + 1024, 1536, 1088)):
        assert attend(lib, q=P(q), out=P(out), ld_q=ld_q, ld_out=ld_out, ws_bytes=0) == L.INVALID_ARG, (out - q, ld_q, ld_out)
    for out, ld_q, ld_out in ((q + end, 512, 512), (q - end, 512, 512), (q + 1024, 1024, 1024),
                              (q - 1024, 1024, 1024),              # side by side in one wide buffer
                              (q + 5120, 1024, 1024),              # from out's second row on, behind q's last one
                              (q + end, 1 << 40, 512), (q + 1024, 2048, 512), (q - 1024, 512, 2048),
                              (q + 1024, 1024, 2048)):
        assert attend(lib, q=P(q), out=P(out), ld_q=ld_q, ld_out=ld_out, ws_bytes=0) == L.WORKSPACE, (out - q, ld_q, ld_out)
    assert attend(lib, q=P(q), out=P(q + 16), ld_q=(1 << 62) + 8, ld_out=(1 << 62) + 8, ws_bytes=0) == L.INVALID_ARG


def test_append_q_out_is_q_or_lies_elsewhere(lib):
    """One unit of a row is read and written by one thread: in place is right with q's own stride alone."""
    from precision_moe_gemm_amd import _lib as L
    rows = dict(q=P(1 << 16), k=P(1 << 17), v=P(1 << 18))

    def refused(**kw):
        """The next check (an empty table of angles) stops what is not refused for its place."""
        s = append(lib, **dict(rows, max_pos=0, **kw))
        assert s in (L.INVALID_ARG, L.SHAPE)
        return s == L.INVALID_ARG

    assert not refused(q_out=P(1 << 16))
    assert refused(q_out=P(1 << 16), ld_qo=1024)
    assert refused(q_out=P((1 << 16) + 16)) and refused(q_out=P((1 << 16) - 16))
    assert refused(q_out=P(1 << 17)) and refused(q_out=P((1 << 17) + 16), ld_qo=512)
    assert refused(q_out=P((1 << 18) - 3 * 1024 + 16))
    assert not refused(q_out=P((1 << 17) - 3 * 1024)) and not refused(q_out=P((1 << 17) + 1536))
    rows = dict(q=P(1 << 16), k=P((1 << 16) + 1024), v=P((1 << 16) + 1536), ld_q=1024, ld_k=1024, ld_v=1024)
    assert not refused(q_out=P(1 << 16), ld_qo=1024)             # the three parts of one projection's rows
    assert refused(q_out=P((1 << 16) + 1024), ld_qo=1024)
    assert not refused(q_out=P(1 << 16), ld_qo=2048, n=1)        # one row has no stride


def test_norm_sum_is_an_input_or_lies_elsewhere(lib):
    """(What is not refused runs on the GPU: the sum in place of either, and beside them in one buffer.)"""
    from precision_moe_gemm_amd import _lib as L
    x, res = 1 << 16, 1 << 17  # 3 rows of 64 elements
    at = dict(x=P(x), res=P(res), y=P(1 << 18), fp8=P(1 << 19), e8=P(1 << 20))
    for base in (x, res):
        for off, ld in ((0, 72), (0, 128), (16, 64), (-16, 64), (128, 64), (-256, 64), (368, 64), (-368, 64), (256, 96)):
            assert norm(lib, **at, sum=P(base + off), ld_sum=ld) == L.INVALID_ARG, (base, off, ld)
    assert norm(lib, **dict(at, res=P(x + 16)), sum=P(x)) == L.INVALID_ARG   # x itself, but part of the residual
    assert norm(lib, **at, sum=P(x + 256), ld_x=128, ld_sum=128) == L.INVALID_ARG


@pytest.mark.skipif("NVFP4_LIB_PATH" in os.environ, reason="this run is the sanitized one")
def test_these_under_asan_ubsan():
    from precision_moe_gemm_amd import build
    env = dict(os.environ, LD_PRELOAD=build.sanitizer_runtime(), NVFP4_LIB_PATH=build.build_sanitized(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_abi_kv_memory_cpu.py"], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=900)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
