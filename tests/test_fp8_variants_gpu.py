"""Kernels of the 8-bit attention that a call is given by its size, and the warp
kernels against the tolerance of their own weights (largest held at 2^15)."""
import numpy as np
import pytest
import torch

from fp8_step import Batch

pytestmark = pytest.mark.gpu


def prefill(lens, new, heads, n_kv, head_dim, dtype, seed=0):
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, dtype=dtype, seed=seed)
    bt.fill()
    q = bt.queries(int(np.sum(new)), heads)
    out = bt.prefill(q, lens, new)
    bt.no_error()
    which = [b for b, c in enumerate(new) for _ in range(c)]
    bt.check(out, q, which, [n - c + i for n, c in zip(lens, new) for i in range(c)], held=15)
    return bt, q, out


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("head_dim", [16, 32])
@pytest.mark.parametrize("rep", [1, 3, 16])
def test_narrow_prefill_of_more_ctas_than_sms(head_dim, rep):
    """bf16 heads of 16 and 32 on two CTAs an SM, which batches with more CTAs
    than SMs get: a query's output is what it is alone, in a batch of one CTA a KV
    head."""
    lens = [1, 40, 65, 200, 17, 300] * 4
    new = [1, 9, 65, 3, 17, 5] * 4
    n_kv = 8
    tile = 8 * (16 // rep)
    busy = n_kv * sum(-(-c // tile) for c in new)
    assert busy > sm_count() >= 1
    bt, q, out = prefill(lens, new, n_kv * rep, n_kv, head_dim, "bf16", seed=rep)
    at = 0
    for b in (0, 3, 4, 5):
        assert n_kv * -(-new[b] // tile) <= sm_count()
    for b, (n, c) in enumerate(zip(lens, new)):
        if b in (0, 3, 4, 5):
            one = Batch([n], n_kv=n_kv, head_dim=head_dim)
            one.d_kp, one.d_vp, one.d_ks, one.d_vs = bt.cache
            one.bt = bt.bt[b:b + 1].contiguous()
            alone = one.prefill(q[at:at + c], [n], [c])
            one.no_error()
            assert torch.equal(alone, out[at:at + c]), b
        at += c


@pytest.mark.parametrize("head_dim,dtype", [(16, "bf16"), (32, "bf16"), (16, "f32"), (32, "f32"),
                                            (64, "f32"), (128, "f32")])
@pytest.mark.parametrize("heads,n_kv", [(8, 4), (9, 3), (16, 1)])
def test_warp_prefill_within_its_own_tolerance(heads, n_kv, head_dim, dtype):
    prefill([300, 1, 129, 64], [37, 1, 129, 20], heads, n_kv, head_dim, dtype, seed=heads)


@pytest.mark.parametrize("n_kv", [1, 2, 4, 5, 6, 7, 16])
@pytest.mark.parametrize("head_dim", [16, 64, 128])
def test_decode_of_many_groups_of_few_heads(n_kv, head_dim):
    """Streaming decodes with one to eight consumer warps a CTA."""
    rng = np.random.default_rng(n_kv)
    lens = rng.integers(1, 2100, size=24)
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, seed=n_kv)
    bt.fill()
    q = bt.queries(24, 2 * n_kv)
    out = bt.decode(q)
    bt.no_error()
    bt.check(out, q, range(24), lens - 1)
