"""Value scales at both ends of their range in one sequence: the softmax's sum
keeps the keys whose values are tiny beside another block's."""
import numpy as np
import pytest
import torch

from fp8_step import Batch

pytestmark = pytest.mark.gpu

STEP = 11  # log2 units by which the large block's keys score higher


def uneven(n, at, head_dim, dtype, small):
    """One sequence of n tokens: block `at`'s values are of magnitude 2^67, the
    others' 0 or of 2^-50, and its first key scores 2^STEP times as high as each
    of theirs (its other keys as they do)."""
    bt = Batch([n], n_kv=1, head_dim=head_dim, dtype=dtype, seed=at)
    k = torch.zeros(n, 1, head_dim)
    v = torch.randn(n, 1, head_dim, generator=bt.g) * small
    lo = 16 * at
    k[lo, 0, 0] = 1.0
    v[lo:lo + 16] = torch.randn(min(16, n - lo), 1, head_dim, generator=bt.g) * 2.0 ** 67
    bt.write([n], [n], k.to(bt.dtype), v.to(bt.dtype))
    assert bt.vs.max() >= 2.0 ** 59 and bt.vs[bt.table[0]].min() <= 2.0 ** -57
    q = torch.zeros(1, 2, head_dim)
    q[..., 0] = STEP * np.log(2) * np.sqrt(head_dim)
    return bt, q.to(bt.dtype)


@pytest.mark.parametrize("small", [0.0, 2.0 ** -50])
@pytest.mark.parametrize("head_dim,dtype", [(16, "bf16"), (64, "bf16"), (128, "bf16"), (64, "f32")])
def test_decode(head_dim, dtype, small):
    """One cluster, one CTA, and several whose parts are joined; the large block
    first, in the middle and last."""
    for n, ctas in ((1000, 0), (1500, 1), (1500, 5), (3200, 0)):
        for at in (0, n // 32, (n - 1) // 16):
            bt, q = uneven(n, at, head_dim, dtype, small)
            out = bt.decode(q, max_ctas=ctas)
            bt.no_error()
            bt.check(out, q, [0], [n - 1])


@pytest.mark.parametrize("small", [0.0, 2.0 ** -50])
@pytest.mark.parametrize("head_dim,dtype", [(16, "bf16"), (64, "bf16"), (128, "bf16"), (64, "f32")])
def test_prefill(head_dim, dtype, small):
    n, c = 1500, 3
    for at in (0, 40, (n - 1) // 16):
        bt, q = uneven(n, at, head_dim, dtype, small)
        q = q.expand(c, -1, -1).contiguous()
        out = bt.prefill(q, [n], [c])
        bt.no_error()
        bt.check(out, q, [0] * c, range(n - c, n), held=4)


@pytest.mark.parametrize("head_dim,dtype", [(16, "bf16"), (64, "bf16"), (128, "bf16"), (64, "f32")])
def test_scales_that_are_no_powers_of_two(head_dim, dtype):
    """A cache that another quantiser wrote, with any positive scales: attended
    and read back at value times scale."""
    import paged_kv_cache_write_gb300 as pkv
    lens = [700, 33, 130]
    bt = Batch(lens, n_kv=2, head_dim=head_dim, dtype=dtype, seed=2)
    bt.fill()
    rng = np.random.default_rng(0)
    for host, dev in ((bt.ks, bt.d_ks), (bt.vs, bt.d_vs)):
        host[:] = (host * rng.uniform(0.5, 2.0, size=host.shape)).astype(np.float32)
        dev.copy_(torch.from_numpy(host))
    q = bt.queries(3, 8)
    for ctas in (0, 1, 7):
        bt.check(bt.decode(q, max_ctas=ctas), q, range(3), [n - 1 for n in lens])
    new = [20, 33, 1]
    q = bt.queries(sum(new), 8)
    out = bt.prefill(q, lens, new)
    bt.check(out, q, [b for b, c in enumerate(new) for _ in range(c)],
             [n - c + i for n, c in zip(lens, new) for i in range(c)], held=4)
    sl, cu = (torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")
              for x in (lens, np.concatenate([[0], np.cumsum(lens)])))
    k, _ = pkv.kv_gather_fp8(*bt.cache, bt.bt, sl, cu, sum(lens), dtype=torch.float32, err=bt.err)
    ref = np.concatenate([bt.rows(b, n)[0] for b, n in enumerate(lens)])
    assert np.array_equal(k.double().cpu().numpy(), ref.astype(np.float32).astype(np.float64))
    bt.no_error()
