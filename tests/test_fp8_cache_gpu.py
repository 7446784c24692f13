"""The 8-bit cache's write and read-back: bytes and scales equal to the
oracle's, for every type, block size and way that tokens arrive in a block."""
import numpy as np
import pytest
import torch

from fp8_step import Batch, f64
from gpu_step import guarded_copy, guarded_empty

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n_kv,head_dim,bs", [(4, 16, 16), (3, 64, 16), (8, 128, 16), (2, 32, 4),
                                              (1, 48, 1), (2, 80, 32), (1, 256, 48), (5, 16, 7)])
def test_prompts_then_steps(dtype, n_kv, head_dim, bs):
    """Whole prompts, then tokens of growing and shrinking size one, two and
    many at a time: blocks begun, filled, crossed and their scales raised."""
    final = [1, bs, 3 * bs + 1, 50, 9, 0]
    bt = Batch(final, n_kv=n_kv, head_dim=head_dim, dtype=dtype, block_size=bs, seed=bs)
    have = np.maximum(0, np.array(final) - np.array([0, 5, 9, 30, 9, 0]))
    t = int(have.sum())
    bt.write(have, have, bt.draw(t), bt.draw(t))
    bt.assert_same_cache()
    step = 0
    while (have < final).any():
        new = np.minimum(np.array(final) - have, [1, 1, 2, 1 + 5 * (step % 4), 1, 1])
        have = have + new
        t = int(new.sum())
        bt.write(have, new, bt.draw(t, 2.0 ** (step % 5 - 1)), bt.draw(t, 2.0 ** (2 - step % 3)))
        bt.assert_same_cache()
        step += 1
    bt.no_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_values(dtype):
    """Zeros, the type's smallest and largest values, values at and beside a
    scale's limit, infinities and NaN; earlier rows that become subnormal or
    vanish when the scale jumps."""
    bt = Batch([16, 16, 16, 16, 4], n_kv=1, head_dim=16, dtype=dtype)
    fi = torch.finfo(bt.dtype)
    k = torch.zeros(52, 1, 16)
    k[0:8] = torch.linspace(-448, 448, 16)              # fits at 2^0 exactly
    k[8] = 448.0 * (1 + fi.eps)                         # just past it: next scale
    k[16:24, :, ::2] = fi.tiny
    k[24, :, 3] = fi.max
    k[32, :, 0] = float("nan")
    k[33, :, 1] = float("inf")
    k[34, :, 2] = -float("inf")
    k[35] = 2.0 ** 68
    # row 48..: all zero
    k = k.to(bt.dtype)
    bt.write([16, 12, 12, 8, 4], [16, 12, 12, 8, 4], k, -k)
    bt.assert_same_cache()
    # one more token each that dwarfs, matches or is dwarfed by the block
    nxt = torch.tensor([0.0, 1e30, 1.0, -2.0 ** 40, 2.0 ** -100]).reshape(5, 1, 1).expand(5, 1, 16).to(bt.dtype)
    bt2 = Batch([16, 16, 16, 16, 5], n_kv=1, head_dim=16, dtype=dtype, seed=1)
    a = bt2.draw(60, 1.0)
    bt2.write([15, 15, 15, 15, 0], [15, 15, 15, 15, 0], a, a * 0.01)
    bt2.write([16, 16, 16, 16, 1], [1, 1, 1, 1, 1], nxt, nxt * 3)
    bt2.assert_same_cache()
    bt.no_error()


def test_many_sequences_and_empty_ones():
    """More sequences than threads, most without a new token, ragged ones
    between; a batch whose tokens end inside a window of 16."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, size=700)
    lens[rng.random(700) < 0.3] = 0
    bt = Batch(lens, n_kv=2, head_dim=32, seed=2)
    new = np.minimum(lens, rng.integers(0, 4, size=700))
    bt.write(lens - new, lens - new, bt.draw(int((lens - new).sum())), bt.draw(int((lens - new).sum())))
    bt.write(lens, new, bt.draw(int(new.sum()), 3.0), bt.draw(int(new.sum()), 0.1))
    bt.assert_same_cache()
    bt.no_error()


def test_rows_behind_the_last_token_are_left():
    bt = Batch([21], n_kv=2, head_dim=64, garbage=0x35)
    bt.write([20], [20], bt.draw(20), bt.draw(20))
    bt.write([21], [1], bt.draw(1, 100.0), bt.draw(1, 100.0))
    bt.assert_same_cache()
    tail = bt.d_kp.view(torch.uint8)[int(bt.table[0, 1]), 5:]
    assert bool((tail == 0x35).all())


def test_same_write_twice_is_the_same_cache():
    bt = Batch([30, 9], n_kv=3, head_dim=64, seed=4)
    bt.fill()
    k, v = bt.draw(2, 5.0), bt.draw(2, 5.0)
    bt.write([30, 9], [1, 1], k, v)
    first = [x.clone().view(torch.uint8) for x in bt.cache]
    bt.write([30, 9], [1, 1], k, v)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(first, bt.cache))
    bt.assert_same_cache()


def test_bad_device_data_is_reported_not_used():
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([20, 7, 18, 4], n_kv=2, head_dim=32)
    before = [x.clone() for x in bt.cache]
    k = guarded_copy(bt.draw(4))

    def write(lens, cu, table=None):
        bt.err.zero_()
        pkv.kv_write_fp8(k, k, bt.bt if table is None else table,
                         guarded_copy(torch.tensor(lens, dtype=torch.int32)),
                         guarded_copy(torch.tensor(cu, dtype=torch.int32)), *bt.cache, err=bt.err)
        torch.cuda.synchronize()
        return int(bt.err.item())

    bad = bt.bt.clone()
    bad[:] = torch.tensor([bt.nb, -1], dtype=torch.int32).cuda()
    D = pkv.DEVERR
    assert write([20, 7, 18, 4], [0, 1, 2, 3, 4], bad) == D["block_id"]
    assert write([200, 33, 1000, 99], [0, 1, 2, 3, 4]) == D["table_width"]
    assert write([-1, 0, -5, -2 ** 31], [0, 1, 2, 3, 4]) == D["length"]
    assert write([0, 0, 0, 0], [0, 1, 2, 3, 4]) == D["length"]       # more new tokens than tokens
    assert write([0, 0, 0, 0], [0, 0, 0, 0, 0]) == D["length"]       # offsets stop short
    assert write([20, 7, 18, 4], [0, 0, 0, 0, 9]) == D["length"]     # offsets past the tokens
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, bt.cache))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n_kv,head_dim,bs", [(4, 16, 16), (3, 64, 16), (8, 128, 16), (1, 48, 5)])
def test_read_back_is_exact(out, n_kv, head_dim, bs):
    lens = [1, 40, 0, 16, 77]
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, block_size=bs, seed=9)
    bt.fill(3.0)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[out]
    shape = (int(cu[-1]), n_kv, head_dim)
    k, v = bt.pkv.kv_gather_fp8(*bt.cache, bt.bt, guarded_copy(torch.from_numpy(bt.lens)),
                                guarded_copy(torch.from_numpy(cu)), int(cu[-1]), dtype=dt,
                                k_out=guarded_empty(shape, dt), v_out=guarded_empty(shape, dt),
                                err=bt.err)
    bt.no_error()
    for b, n in enumerate(lens):
        rk, rv = bt.rows(b, n)
        assert np.array_equal(f64(k[cu[b]:cu[b + 1]]), rk)
        assert np.array_equal(f64(v[cu[b]:cu[b + 1]]), rv)
    assert k.dtype == dt


def test_read_back_reports_bad_data_and_reads_zeros():
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([20, 20], n_kv=2, head_dim=32)
    bt.fill()
    D = pkv.DEVERR

    def read(lens, cu, total, table):
        bt.err.zero_()
        k, _ = pkv.kv_gather_fp8(*bt.cache, table, guarded_copy(torch.tensor(lens, dtype=torch.int32)),
                                 guarded_copy(torch.tensor(cu, dtype=torch.int32)), total, err=bt.err)
        torch.cuda.synchronize()
        return int(bt.err.item()), k

    bad = bt.bt.clone()
    bad[0, 1] = bt.nb
    e, k = read([20, 20], [0, 20, 40], 40, bad)
    assert e == D["block_id"] and not k[16:20].any() and bool(k[:16].any())
    e, k = read([20, 20], [0, 20, 44], 44, bt.bt)
    assert e == D["length"] and not k[40:].any()
    e, _ = read([20, 20], [0, 20, 40], 44, bt.bt)
    assert e == D["length"]
    e, _ = read([40, 20], [0, 40, 60], 60, bt.bt)
    assert e == D["table_width"]


def test_blocks_are_copied_with_copy_blocks():
    """Copy-on-write of a shared block: pools as bf16 of half the width,
    scales as fp32 blocks of one token."""
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([40, 3], n_kv=4, head_dim=32, spare=4)
    bt.fill()
    src, dst = int(bt.table[0, 1]), next(i for i in range(bt.nb) if i not in bt.table[:, :3].ravel())
    pairs = guarded_copy(torch.tensor([[src, dst]], dtype=torch.int32))
    nb = bt.nb
    pkv.copy_blocks(bt.d_kp.view(torch.bfloat16).view(nb, 16, 4, 16),
                    bt.d_vp.view(torch.bfloat16).view(nb, 16, 4, 16), pairs, err=bt.err)
    pkv.copy_blocks(bt.d_ks.view(nb, 1, 1, 4), bt.d_vs.view(nb, 1, 1, 4), pairs, err=bt.err)
    bt.no_error()
    for x in (bt.kp, bt.vp, bt.ks, bt.vs):
        x[dst] = x[src]
    bt.assert_same_cache()


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB: blocks at its end are written, read back
    and attended where they are."""
    nb = 280_000  # x 16 KB = 4.6 GB a pool
    shape = (nb, 16, 8, 128)
    import paged_kv_cache_write_gb300 as pkv
    kp, vp = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones(nb, 8, device="cuda") for _ in range(2))
    bt = torch.tensor([[nb - 1, 3], [nb - 2, 270_000]], dtype=torch.int32, device="cuda")
    sl = torch.tensor([20, 32], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20, 52], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.randn(52, 8, 128, device="cuda").to(torch.bfloat16)
    v = torch.randn(52, 8, 128, device="cuda").to(torch.bfloat16)
    pkv.kv_write_fp8(k, v, bt, sl, cu, kp, vp, ks, vs, err=err)
    kb, vb = pkv.kv_gather_fp8(kp, vp, ks, vs, bt, sl, cu, 52, dtype=torch.float32, err=err)
    for got, x in ((kb, k), (vb, v)):
        amax = x.float().abs().amax()
        assert bool(((got - x.float()).abs() <= x.float().abs() * 2 ** -4 + amax * 2 ** -18).all())
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    out = pkv.paged_attention_decode_fp8(q, kp, vp, ks, vs, bt, sl, 0.1, 32, err=err)
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    pre = pkv.paged_attention_prefill_fp8(q, one, kp, vp, ks, vs, bt, sl, 0.1, 1, 32, err=err)
    assert int(err.item()) == 0
    for b in range(2):
        kk, vv = kb[cu[b]:cu[b + 1]].double(), vb[cu[b]:cu[b + 1]].double()
        p = torch.softmax(0.1 * torch.einsum("hd,nhd->hn", q[b].double(), kk), -1)
        ref = torch.einsum("hn,nhd->hd", p, vv)
        # 2^-8 for the output's rounding, 2^-9 of the values' mean magnitude for the weights
        tol = 2 ** -8 * ref.abs() + 2 ** -9 * torch.einsum("hn,nhd->hd", p, vv.abs())
        assert bool(((out[b].double() - ref).abs() <= tol).all())
        assert bool(((pre[b].double() - ref).abs() <= tol).all())
