"""Limits of the 8-bit cache and token-tree calls that the host checks, and their RoPE angles on the
host.  No GPU: every call here fails before any CUDA call."""
import pytest

from tests.test_abi_fp8_tree import call, lib  # noqa: F401 (lib is the fixture)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw", [dict(B=32768, Hkv=32768), dict(B=65535, Hkv=32767)])
def test_read_of_too_many_heads(lib, kw, paged):  # noqa: F811
    """B * Hkv at 2^30 and above is past the limits, not a failed launch."""
    assert call(lib, "read", paged, Lout=1, pages=16, **kw) == -2
    assert b"too large" in lib.csattn_last_error()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("op", ["append", "decode", "tree"])
def test_rope_bases_below_one(lib, op, paged):  # noqa: F811
    """Angles past the range in which they are reduced exactly are refused; those within go on (to
    the check of something else)."""
    for kw in (dict(base=1e-3), dict(base=1e-3, d=128), dict(base=1e-30)):
        assert call(lib, op, paged, **kw) == -2
        assert b"RoPE" in lib.csattn_last_error()
    if op != "append":
        assert call(lib, op, paged, base=0.5, ws=None) == -5
        assert call(lib, op, paged, base=0.01, ws=None) == -5
