"""8-bit calls beside others that start early, without a wait between them:
what one leaves is what the next one reads."""
import numpy as np
import pytest
import torch

from fp8_step import Batch
from gpu_step import guarded_copy, guarded_empty

pytestmark = pytest.mark.gpu


def ints(x):
    return guarded_copy(torch.as_tensor(np.asarray(x, dtype=np.int32)))


@pytest.mark.parametrize("n,tokens,heads,n_kv,head_dim", [(64, 512, 32, 8, 64), (40, 1600, 16, 4, 128),
                                                          (3, 96, 9, 3, 64)])
def test_read_back_into_a_bf16_cache_then_planned_decode(n, tokens, heads, n_kv, head_dim):
    """A planned decode of the bf16 cache reads its first blocks before it waits
    for the kernel before it: here the read-back that fills them."""
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([tokens] * n, n_kv=n_kv, head_dim=head_dim, seed=n)
    total, blocks = n * tokens, n * tokens // 16
    sl, cu = ints([tokens] * n), ints(np.arange(n + 1) * tokens)
    table = ints(np.arange(blocks).reshape(n, -1))
    k_pool, v_pool = (guarded_empty((blocks, 16, n_kv, head_dim), torch.bfloat16) for _ in range(2))
    rows = [p.view(total, n_kv, head_dim) for p in (k_pool, v_pool)]
    q = guarded_copy(bt.queries(n, heads))
    scale = 1.0 / np.sqrt(head_dim)
    ws = guarded_empty((pkv.decode_workspace_bytes(n, heads, head_dim, tokens),), torch.uint8)
    own = guarded_empty((pkv.decode_workspace_bytes(n, heads, head_dim, tokens),), torch.uint8)
    out = guarded_empty(q.shape, q.dtype)
    for step in range(8):
        x = [guarded_copy(bt.draw(total)) for _ in range(2)]
        pkv.kv_write_fp8(*x, bt.bt, sl, cu, *bt.cache, err=bt.err)
        for p in (k_pool, v_pool):
            p.fill_(float("nan"))
        pkv.decode_plan(k_pool, sl, heads, tokens // 16, tokens, workspace=ws, err=bt.err)
        torch.cuda.synchronize()
        pkv.kv_gather_fp8(*bt.cache, bt.bt, sl, cu, total, k_out=rows[0], v_out=rows[1], err=bt.err)
        pkv.paged_attention_decode_planned(q, k_pool, v_pool, table, sl, scale, tokens, workspace=ws,
                                           out=out, err=bt.err)
        torch.cuda.synchronize()
        ref = pkv.paged_attention_decode(q, k_pool, v_pool, table, sl, scale, tokens, workspace=own,
                                         err=bt.err)
        assert torch.equal(out, ref) and bool(out.isfinite().all()), step
    bt.no_error()
