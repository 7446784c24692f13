"""Prefill where weights outgrow their reference time and again: tiles whose
weights are computed, found past f16's range and computed again."""
import numpy as np
import pytest
import torch

from fp8_step import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("head_dim", [32, 64, 128])
@pytest.mark.parametrize("step", [13, 40])
def test_scores_that_grow_from_tile_to_tile(head_dim, dtype, step):
    """Keys in runs of 64 whose scores are `step` log2 units above the run
    before, for every other query head; the others' stay within one unit (rows
    that keep their reference beside rows that move it).  Repeated calls give the
    same bits."""
    n, heads = 640, 4
    bt = Batch([n], n_kv=1, head_dim=head_dim, dtype=dtype, seed=step)
    k = torch.randn(n, 1, head_dim, generator=bt.g) * 0.05
    k[:, 0, 0] = (torch.arange(n) // 64).float()
    k[:, 0, 1] = torch.rand(n, generator=bt.g)
    bt.write([n], [n], k.to(bt.dtype), bt.draw(n))
    q = torch.randn(n, heads, head_dim, generator=bt.g) * 0.05
    q[..., :2] = 0
    q[:, ::2, 0] = step * np.log(2) * np.sqrt(head_dim)
    q[:, 1::2, 1] = np.log(2) * np.sqrt(head_dim)
    q = q.to(bt.dtype)
    outs = [bt.prefill(q, [n], [n]) for _ in range(12)]
    bt.no_error()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    bt.check(outs[0], q, [0] * n, range(n), held=4)
