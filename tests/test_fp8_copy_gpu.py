"""Copy-on-write of 8-bit blocks for any number of KV heads."""
import pytest
import torch

from fp8_step import Batch
from gpu_step import guarded_copy

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_kv", [1, 2, 3, 5, 8, 10])
def test_a_shared_block_is_copied_then_written(n_kv):
    """Two sequences share a block that is half full; one copies it (bytes and
    scales) and writes its next token there, which raises the copy's scales."""
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([24, 24], n_kv=n_kv, head_dim=64, spare=4)
    bt.fill()
    src, dst = int(bt.table[0, 1]), next(i for i in range(bt.nb) if i not in bt.table)
    pairs = guarded_copy(torch.tensor([[src, dst], [src, -1], [bt.nb, dst]], dtype=torch.int32))
    nb = bt.nb
    pkv.copy_blocks(bt.d_kp.view(torch.bfloat16).view(nb, 16, n_kv, 32),
                    bt.d_vp.view(torch.bfloat16).view(nb, 16, n_kv, 32), pairs[:1])
    pkv.copy_blocks(bt.d_ks.view(nb, 1, 1, n_kv), bt.d_vs.view(nb, 1, 1, n_kv), pairs, err=bt.err)
    torch.cuda.synchronize()
    assert int(bt.err.item()) == pkv.DEVERR["block_id"]  # (the second and third pair)
    bt.err.zero_()
    for x in (bt.kp, bt.vp, bt.ks, bt.vs):
        x[dst] = x[src]
    bt.assert_same_cache()
    bt.table[1, :] = [bt.table[0, 0], dst]
    bt.bt.copy_(torch.from_numpy(bt.table))
    bt.write([24, 25], [0, 1], bt.draw(1, 50.0), bt.draw(1, 50.0))
    bt.no_error()
    bt.assert_same_cache()


@pytest.mark.parametrize("shape,dtype", [((40, 1, 1, 3), torch.float32), ((33, 5, 3, 1), torch.float32),
                                         ((64, 3, 1, 2), torch.bfloat16), ((20, 7, 5, 30), torch.bfloat16),
                                         ((9, 1, 1, 1), torch.float32), ((50, 16, 3, 1000), torch.bfloat16)])
def test_blocks_of_any_whole_words(shape, dtype):
    """Blocks of whole and of no whole 16-byte words, bit for bit."""
    import paged_kv_cache_write_gb300 as pkv
    g = torch.Generator().manual_seed(shape[0])
    k, v = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
    ids = torch.randperm(shape[0], generator=g)
    n = shape[0] // 2
    pairs = torch.stack([ids[:n], ids[n:2 * n]], dim=1).to(torch.int32)
    dk, dv = guarded_copy(k), guarded_copy(v)
    pkv.copy_blocks(dk, dv, guarded_copy(pairs))
    for x in (k, v):
        x[ids[n:2 * n]] = x[ids[:n]]
    assert torch.equal(dk.cpu(), k) and torch.equal(dv.cpu(), v)
