"""Bad device data in the 8-bit prefill: what is reported is the same for every
type, head width and batch size, whichever kernel the call goes to."""
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


@pytest.mark.parametrize("head_dim,dtype,n", PATHS)
def test_any_block_id_out_of_range_is_reported(head_dim, dtype, n):
    """-1, the usual filler of a table, is a bad id where it stands for a block
    that the sequence holds; it is read as zeros like any other."""
    import paged_kv_cache_write_gb300 as pkv
    bt, q, lens, new = batch(head_dim, dtype, n)
    good = bt.prefill(q, lens, new)
    bt.no_error()
    seen = []
    for bad in (-7, -1, bt.nb, -2 ** 31, 2 ** 31 - 1):
        bt.bt[1, 1] = bad
        out = bt.prefill(q, lens, new)
        torch.cuda.synchronize()
        assert int(bt.err.item()) == pkv.DEVERR["block_id"], bad
        assert torch.equal(out[:6], good[:6]) and torch.equal(out[12:], good[12:])
        seen.append(out[6:12].clone())
        bt.err.zero_()
    assert all(torch.equal(x, seen[0]) for x in seen) and not torch.equal(seen[0], good[6:12])


@pytest.mark.parametrize("head_dim,dtype,n", PATHS)
def test_filler_behind_a_sequences_blocks_is_not_reported(head_dim, dtype, n):
    bt, q, lens, new = batch(head_dim, dtype, n)
    good = bt.prefill(q, lens, new)
    wide = np.full((n, 9), -1, dtype=np.int32)
    wide[:, :3] = bt.table
    bt.bt = guarded_copy(torch.from_numpy(wide))
    assert torch.equal(bt.prefill(q, lens, new), good)
    bt.no_error()
