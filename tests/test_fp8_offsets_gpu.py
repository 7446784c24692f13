"""Offsets of the 8-bit prefill and write that disagree with their arguments."""
import numpy as np
import pytest
import torch

from fp8_step import Batch
from gpu_step import guarded_copy, guarded_empty

pytestmark = pytest.mark.gpu

# (head_dim, type, sequences): tcgen05 with an ordered and with a plain grid
# (more than 512 sequences), warp-level products
PATHS = [(64, "bf16", 3), (128, "bf16", 3), (64, "bf16", 600), (128, "bf16", 600), (16, "bf16", 3),
         (32, "bf16", 3), (64, "f32", 3), (128, "f32", 3)]


def ints(x):
    return guarded_copy(torch.as_tensor(np.asarray(x, dtype=np.int32)))


def batch(head_dim, dtype, n):
    """n sequences of 40 tokens and the last 6 of each as a chunk."""
    bt = Batch([40] * n, n_kv=1, head_dim=head_dim, dtype=dtype, seed=n)
    bt.fill()
    return bt, bt.queries(6 * n, 2), [40] * n, [6] * n

# offsets of 3 chunks over 18 query rows that disagree with the rows, with each
# other or with the largest chunk (6); the chunks that hold all the same
@pytest.mark.parametrize("cu,good", [([0, 6, 12, 16], (0, 1)),           # stop short of the rows
                                     ([0, 6, 12, 30], (0, 1)),           # go past them
                                     ([12, 6, 12, 18], (1, 2)),          # go back
                                     ([0, 6, 15, 18], (0, 2)),           # a chunk longer than max_q_len
                                     ([0, 2 ** 31 - 1, 12, 18], (2,)),
                                     ([0, 1 << 20, 1 << 20, 1 << 20], ()),
                                     ([-6, 0, 12, 18], (2,))])
@pytest.mark.parametrize("head_dim,dtype,n", PATHS)
def test_offsets_that_disagree_are_reported(head_dim, dtype, n, cu, good):
    """Rows that belong to no chunk are left as they were."""
    import paged_kv_cache_write_gb300 as pkv
    bt, q, lens, new = batch(head_dim, dtype, n)
    ref = bt.prefill(q, lens, new)
    bt.no_error()
    # the last three sequences of the batch, the others without a query
    table = bt.bt.flip(0).contiguous()
    cu = ints([cu[0]] * (n - 3) + cu)
    out = guarded_empty((18, 2, head_dim), bt.dtype)
    out.fill_(7.0)
    q3 = guarded_copy(q[:18])
    pkv.paged_attention_prefill_fp8(q3, cu, *bt.cache, table, ints(lens), 1.0 / np.sqrt(head_dim), 6,
                                    40, out=out, err=bt.err)
    torch.cuda.synchronize()
    assert int(bt.err.item()) == pkv.DEVERR["length"]
    bt.err.zero_()
    want = guarded_empty((18, 2, head_dim), bt.dtype)
    pkv.paged_attention_prefill_fp8(q3, ints([0] * (n - 3) + [0, 6, 12, 18]), *bt.cache, table,
                                    ints(lens), 1.0 / np.sqrt(head_dim), 6, 40, out=want, err=bt.err)
    bt.no_error()
    at = cu[-4:].tolist()
    owned = torch.zeros(18, dtype=torch.bool, device="cuda")
    for i in range(3):
        lo, hi = max(0, at[i]), min(18, at[i + 1])
        owned[lo:hi] = True
        if i in good and (lo, hi) == (6 * i, 6 * i + 6):
            assert torch.equal(out[lo:hi], want[lo:hi]), i
    assert bool((out[~owned] == 7.0).all())
    assert ref.shape[0] == 6 * n


@pytest.mark.parametrize("n", [4, 700])
def test_write_reports_sequences_past_the_tokens(n):
    """The last sequences' tokens are not among those given: the others' are
    written and the loss is reported."""
    import paged_kv_cache_write_gb300 as pkv
    bt, ref = (Batch([20] * n, n_kv=2, head_dim=32, seed=1) for _ in range(2))
    k = guarded_copy(bt.draw(3))
    lens = ints([20] * n)
    for cu in ([0, 1, 2, 3] + [4] * (n - 3), [0, 1, 2, 3] + [2 ** 31 - 1] * (n - 3)):
        bt.err.zero_()
        pkv.kv_write_fp8(k, k, bt.bt, lens, ints(cu), *bt.cache, err=bt.err)
        torch.cuda.synchronize()
        assert int(bt.err.item()) == pkv.DEVERR["length"]
    pkv.kv_write_fp8(k, k, ref.bt, lens, ints([0, 1, 2, 3] + [3] * (n - 3)), *ref.cache, err=ref.err)
    ref.no_error()
    for x, y in zip(bt.cache, ref.cache):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
