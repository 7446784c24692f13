"""The 4-bit writes under head scales that the cache's format does not have: reported, and
the head's rows left as they were."""
import numpy as np
import pytest
import torch

from fp4_step import Batch, f64, ints
from gpu_step import check_canaries, guarded_copy
from test_norm_rope_gpu import Step, rows_out

pytestmark = pytest.mark.gpu

BAD = [0.75, 3.0, 1.0 + 2.0 ** -23, 0.0, -1.0, 2.0 ** -61, 2.0 ** 61, 1e-40, float("nan"), float("inf")]


def expect(bt, slots, k, v, k_bad, v_bad):
    """The oracle's cache after a write whose K / V scales of some heads are bad."""
    before = [x.copy() for x in (bt.kp, bt.kg, bt.vp, bt.vg)]
    bt.take(slots, f64(k), f64(v))
    for x, old, heads in zip((bt.kp, bt.kg, bt.vp, bt.vg), before, (k_bad, k_bad, v_bad, v_bad)):
        x[:, heads] = old[:, heads]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", BAD)
def test_write(bad, dtype):
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([40], n_kv=3, head_dim=32, dtype=dtype)
    bt.d_ks[1] = bad
    bt.d_vs[2] = bad
    k, v = bt.draw(40), bt.draw(40)
    slots = bt.slots([40], [40])
    pkv.kv_write_fp4(guarded_copy(k), guarded_copy(v), ints(slots, np.int64), *bt.cache, err=bt.err)
    check_canaries()
    assert int(bt.err.item()) == pkv.DEVERR["scale"]
    expect(bt, slots, k, v, [1], [2])
    bt.assert_same_cache()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_rope_write(dtype, interleaved):
    """The queries come out as ever."""
    import paged_kv_cache_write_gb300 as pkv
    s = Step(21, 6, 3, 64, 64, dtype, interleaved=interleaved, seed=5)
    bt = Batch([21], n_kv=3, head_dim=64, dtype=dtype)
    bt.d_ks[0] = 1.5
    slots = bt.slots([21], [21])
    q, k = rows_out(s)
    got = pkv.qk_norm_rope_write_fp4(s.q, s.k, s.v, *s.args, ints(slots, np.int64), *bt.cache, **s.kw_args,
                                     err=bt.err)
    check_canaries()
    assert int(bt.err.item()) == pkv.DEVERR["scale"] and torch.equal(q, got)
    expect(bt, slots, k, s.v, [0], [])
    bt.assert_same_cache()


@pytest.mark.parametrize("g", [2.0 ** -60, 2.0 ** 60])
def test_the_ends_of_the_range_are_scales(g):
    bt = Batch([20], n_kv=2, head_dim=16, scale=g)
    k, v = (bt.draw(20).float() * g).to(bt.dtype), (bt.draw(20).float() * g).to(bt.dtype)
    bt.write(bt.slots([20], [20]), k, v)
    bt.no_error()
    bt.assert_same_cache()
