"""The 8-bit kernels' failure path, exercised without a fault: a warp's wait for
a phase that nothing completes runs out, every lane learns of it, and the
context keeps working."""
import time

import pytest
import torch

import paged_kv_cache_write_gb300 as pkv
from fp8_step import Batch

pytestmark = pytest.mark.gpu


def test_a_warp_gives_up_as_one():
    """Half of the warp's lanes wait for a complete phase, half for one that never
    is.  (After another thread gave up the wait ends at once: the kernels' own
    limit is 2 s.)"""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    pkv.selftest_bounded_wait_fp8(err, polls=64)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert int(err.item()) == pkv.DEVERR["timeout"]
    bt = Batch([5, 40, 300], n_kv=4, head_dim=64, seed=3)
    bt.fill()
    q = bt.queries(3, 16)
    for ctas in (0, 3):
        out = bt.decode(q, max_ctas=ctas)
        bt.no_error()
        bt.check(out, q, range(3), [4, 39, 299])
