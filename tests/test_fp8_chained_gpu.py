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


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("n,head_dim,dtype", [(5, 64, "bf16"), (5, 32, "bf16"), (5, 128, "f32"),
                                              (700, 64, "bf16"), (40, 128, "bf16")])
def test_lengths_offsets_and_tables_written_by_the_kernel_before(n, head_dim, dtype, captured):
    """Each call follows the kernels that write its lengths, offsets and table
    without a wait; between calls they hold zeros."""
    import paged_kv_cache_write_gb300 as pkv
    rng = np.random.default_rng(n)
    most = 40 if n > 100 else 300
    lens = rng.integers(3, most, size=(3, n))
    lens[2][::2] = most
    bt = Batch(lens.max(axis=0), n_kv=2, head_dim=head_dim, dtype=dtype, seed=n)
    bt.fill()
    # three batches: the sequences in another order each, the first with a chunk of 1 - 3 queries
    batches = []
    for i in range(3):
        p = rng.permutation(n)
        have, new = lens[i][p], np.where(np.arange(n) == 0, 1 + i, 1)
        batches.append([ints(x) for x in (have, np.concatenate([[0], np.cumsum(new)]),
                                          np.concatenate([[0], np.cumsum(have)]), bt.table[p])])
    total = [int(x.sum()) for x in lens]
    sl, cu, full, table = (guarded_empty(x.shape, x.dtype) for x in batches[0])
    qs = [guarded_copy(bt.queries(n + i, 8)) for i in range(3)]
    ws = guarded_empty((pkv.decode_fp8_workspace_bytes(n, 8, head_dim, most),), torch.uint8)
    outs = [[guarded_empty((m, h, head_dim), bt.dtype)
             for m, h in ((n, 8), (n + i, 8), (total[i], 2), (total[i], 2))] for i in range(3)]
    s = 1.0 / np.sqrt(head_dim)

    def step(i, between=lambda: None):
        dec, pre, kb, vb = outs[i]
        for x in outs[i]:
            x.zero_()

        def written(last):
            """The batch's integers, `last` by the kernel right before the call."""
            pairs = sorted(zip((sl, cu, full, table), batches[i]), key=lambda xy: xy[0] is last)
            for x, _ in pairs:
                torch.mul(x, 0, out=x)
            for x, y in pairs:
                torch.add(y, 0, out=x)
            between()

        for last in (sl, table):
            written(last)
            pkv.paged_attention_decode_fp8(qs[i][:n], *bt.cache, table, sl, s, most, out=dec,
                                           workspace=ws, err=bt.err)
            between()
        for last in (sl, cu, table):
            written(last)
            pkv.paged_attention_prefill_fp8(qs[i], cu, *bt.cache, table, sl, s, 3, most, out=pre,
                                            err=bt.err)
            between()
        for last in (sl, full, table):
            written(last)
            pkv.kv_gather_fp8(*bt.cache, table, sl, full, total[i], k_out=kb, v_out=vb, err=bt.err)
            between()

    sl.zero_(), cu.zero_(), full.zero_(), table.zero_()
    ref = []
    for i in range(3):
        step(i, torch.cuda.synchronize)
        ref.append([x.clone() for x in outs[i]])
    bt.no_error()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            for i in range(3):
                step(i)
    for _ in range(10):
        if captured:
            graph.replay()
        else:
            for i in range(3):
                step(i)
        torch.cuda.synchronize()
        for i in range(3):
            assert all(torch.equal(x, y) for x, y in zip(outs[i], ref[i])), i
    bt.no_error()
