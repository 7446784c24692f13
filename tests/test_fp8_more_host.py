"""More refusals of the 8-bit entries (host checks that run before any launch
and never touch a GPU)."""
import pytest

FAKE = 0x10000  # a 16-byte-aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_write_gb300 import build
    build.build()
    import paged_kv_cache_write_gb300 as m
    return m


def test_selftest_bounded_wait_refusals(pkv):
    assert pkv.lib.pkv_selftest_bounded_wait_fp8(0, FAKE, None) == 5
    assert pkv.lib.pkv_selftest_bounded_wait_fp8(64, None, None) == 1
