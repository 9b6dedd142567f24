"""Refusals of the cache and norm operators that concern where their operands lie: found on the host, before
any launch (no GPU here)."""
from tests.test_abi_kv_cpu import P, append, attend, cache, lib, norm  # noqa: F401  (lib: the fixture)


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
