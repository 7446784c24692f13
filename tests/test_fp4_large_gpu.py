"""The norm, rotation and 4-bit entries at sizes past a grid's and a 32-bit offset's ends."""
import numpy as np
import pytest
import torch

from fp4_step import Batch, f64, ints
from gpu_step import check_canaries
from oracle import paged_fp4
from test_norm_rope_gpu import bound, table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head_dim,dtype", [(16, "bf16"), (64, "bf16"), (32, "f32")])
def test_more_sequences_than_a_grid_is_deep(head_dim, dtype):
    """66,000 sequences: prefill goes in slices of 65,535, a stream's plan past 8,191 lies in
    the workspace."""
    n = 66_000
    rng = np.random.default_rng(head_dim)
    lens = rng.integers(0, 3, size=n)
    lens[[0, 65_534, 65_535, n - 1]] = 2
    bt = Batch(lens, n_kv=1, head_dim=head_dim, dtype=dtype, seed=1)
    bt.fill()
    rows = np.unique(np.concatenate([rng.integers(0, n, size=100), [0, 65_533, 65_534, 65_535, 65_536, n - 1]]))
    q = bt.queries(n, 2)
    for ctas in (0, 100):
        out = bt.decode(q, max_ctas=ctas)
        bt.no_error()
        bt.check(out[rows], q[rows], rows, lens[rows] - 1)
        assert not out[torch.from_numpy(lens == 0).cuda()].any()
    first = np.concatenate([[0], np.cumsum(lens)])[:-1]
    q = bt.queries(int(lens.sum()), 2)
    out = bt.prefill(q, lens, lens)
    bt.no_error()
    for i in range(2):  # the sampled sequences' first and second queries
        which = rows[lens[rows] > i]
        bt.check(out[first[which] + i], q[first[which] + i], which, [i] * len(which))


def test_rows_past_2_to_31_elements():
    """A projection's output, queries out and slots whose elements pass 32-bit offsets."""
    import paged_kv_cache_write_gb300 as pkv
    T, heads, n_kv, hd = 600_000, 28, 2, 128
    assert T * heads * hd > 1 << 31
    torch.manual_seed(0)
    qkv = torch.empty(T, (heads + 2 * n_kv) * hd, dtype=torch.bfloat16, device="cuda").normal_()
    q, k, v = (x.unflatten(1, (-1, hd)) for x in qkv.split([heads * hd, n_kv * hd, n_kv * hd], dim=1))
    cs = table(1000, hd)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 1000
    w = [torch.rand(hd, device="cuda").add(0.5).bfloat16() for _ in range(2)]
    nb = (T + 15) // 16
    slots = (nb * 16 - 1) - torch.arange(T, device="cuda")  # backwards
    pools = [torch.zeros(nb, n_kv, 16, hd // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    groups = [torch.zeros(nb, n_kv, 16, hd // 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
              for _ in range(2)]
    scales = [torch.full((n_kv,), 0.25, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.qk_norm_rope_write_fp4(q, k, v, cs.cuda(), pos, slots, *pools, *groups, *scales, q_weight=w[0],
                                     k_weight=w[1], eps=1e-5, err=err)
    q2, k2 = pkv.qk_norm_rope(q, k, cs.cuda(), pos, q_weight=w[0], k_weight=w[1], eps=1e-5, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, q2)
    edge = (1 << 31) // (heads * hd)
    for t in (0, 1, edge - 1, edge, edge + 1, (1 << 31) // qkv.shape[1], T - 2, T - 1):
        for x, y, wt in ((q, out, w[0]), (k, k2, w[1])):
            ref, tol = bound(f64(x[t:t + 1]), f64(wt), 1e-5, cs.numpy(), [t % 1000], False, torch.bfloat16)
            assert np.all(np.abs(f64(y[t:t + 1]) - ref) <= tol), t
        at = nb * 16 - 1 - t
        for x, p, g in ((k2, pools[0], groups[0]), (v, pools[1], groups[1])):
            codes, s8 = paged_fp4.quantise(f64(x[t:t + 1]), np.full(n_kv, 0.25))
            assert np.array_equal(p[at // 16, :, at % 16].cpu().numpy(), codes[0])
            assert np.array_equal(g.view(torch.uint8)[at // 16, :, at % 16].cpu().numpy(), s8[0])
    check_canaries()
