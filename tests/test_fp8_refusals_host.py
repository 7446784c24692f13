"""More refusals of the 8-bit entries (host checks that run before any launch
and never touch a GPU)."""
import ctypes

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


def test_attention_refuses_more_kv_heads_than_its_grids_hold(pkv):
    for n_kv, status in ((65535, 7), (65536, 5), (65537, 5), (1 << 20, 5)):
        # (65,535 goes on to the next check: 17 query heads a KV head are refused)
        d = pkv.PoolDesc(8, 16, n_kv, 64, pkv.PKV_FP8_E4M3)
        by = ctypes.byref(d)
        assert pkv.lib.pkv_paged_attention_decode_fp8(
            FAKE, 1, 2, 17 * n_kv, FAKE, FAKE, FAKE, FAKE, by, FAKE, 4, FAKE, 64, 0.1, 0, FAKE, FAKE,
            1 << 60, None, None) == status
        assert pkv.lib.pkv_paged_attention_prefill_fp8(
            FAKE, 1, FAKE, 2, 10, 8, 17 * n_kv, FAKE, FAKE, FAKE, FAKE, by, FAKE, 4, FAKE, 64, 0.1,
            FAKE, None, None) == status


def test_copy_blocks_takes_rows_of_whole_4_byte_words(pkv):
    def copy(**kw):
        d = pkv.PoolDesc(**{**dict(num_blocks=8, block_size=1, n_kv=1, head_dim=3, dtype=0), **kw})
        return pkv.lib.pkv_copy_blocks(FAKE, FAKE, ctypes.byref(d), FAKE, 0, None, None)
    assert copy() == 0 and copy(head_dim=1) == 0 and copy(dtype=1, head_dim=2) == 0
    assert copy(dtype=1) == 4  # bf16 rows of 6 bytes
