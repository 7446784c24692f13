"""Writing a 4-bit cache and reading it back, code by code against the float64
oracle."""
import numpy as np
import pytest
import torch

from fp4_step import Batch, f64, ints
from gpu_step import check_canaries, guarded_copy, guarded_empty
from oracle import paged_fp4

pytestmark = pytest.mark.gpu


def gather(bt, lens, dtype=None, err=None):
    cu = np.concatenate([[0], np.cumsum(lens)])
    shape = (int(cu[-1]), bt.n_kv, bt.hd)
    out = bt.pkv.kv_gather_fp4(*bt.cache, bt.bt, ints(lens), ints(cu), shape[0],
                               k_out=guarded_empty(shape, dtype or bt.dtype),
                               v_out=guarded_empty(shape, dtype or bt.dtype),
                               err=bt.err if err is None else err)
    check_canaries()
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n_kv,head_dim,block_size", [(1, 16, 16), (4, 16, 16), (3, 32, 16), (8, 64, 16),
                                                      (5, 64, 4), (8, 128, 16), (2, 80, 1), (3, 96, 32),
                                                      (32, 128, 16), (2, 256, 16)])
def test_write_then_read_back(n_kv, head_dim, block_size, dtype):
    lens = [1, 15, 0, 16, 17, 100]
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, block_size=block_size, dtype=dtype, seed=head_dim)
    bt.fill()
    bt.assert_same_cache()
    for step in range(2):  # some sequences take one token or several more, others none
        new = [1, 0, 0, 3, 17, 40][:: 1 if step else -1]
        new = [min(a, b) for a, b in zip(new, lens)]
        t = sum(new)
        bt.write(bt.slots(lens, new), bt.draw(t, 4.0), bt.draw(t, 0.1))
        bt.assert_same_cache()
    for out in (torch.float32, torch.bfloat16):
        k, v = gather(bt, lens, out)
        rows = [bt.rows(b, n) for b, n in enumerate(lens)]
        # (6 significand bits times a power of two: a bf16 number)
        assert np.array_equal(f64(k), np.concatenate([r[0] for r in rows]))
        assert np.array_equal(f64(v), np.concatenate([r[1] for r in rows]))
    bt.no_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_border_between_codes(dtype):
    """Elements at, just below and just above the borders of e2m1, under each scale; and
    groups whose largest element puts the scale at, below and above the borders of
    e4m3."""
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    scales = paged_fp4.E4M3[1:127]  # 2^-9 .. 448

    def near(x):
        x = torch.tensor(x, dtype=torch.float64).to(t)
        i = x.view(torch.int32 if t == torch.float32 else torch.int16)
        return [float((i + d).view(t)) for d in (-1, 0, 1)]

    groups = []
    for s in scales:
        for m in mid:
            below, at, above = near(m * s)
            groups.append([6 * s, below, -below, at, -at, above, -above, 0.0, -0.0, s, -s] + [1.5 * s] * 5)
    for a, b in zip(scales, paged_fp4.E4M3[2:127]):
        for top in near(6 * (a + b) / 2):
            groups.append([top] + [top * f for f in (0.9, -0.5, 0.04, 0.24, 0.26)] + [0.0] * 10)
    groups += [[0.0] * 16, [-0.0] * 16, [1e-5] * 16, [2.0 ** -9 * 3] * 16, [2.0 ** -9 * 3.01] + [0.0] * 15]
    groups += [[x] + [1.0] * 15 for x in (2687.0, 2688.0, 2689.0, 1e9, -3e38)]
    x = torch.tensor(groups, dtype=torch.float64).to(t)
    n_kv, hd = 2, 64
    pad = -len(x) % (n_kv * hd // 16)
    x = torch.cat([x, x[:pad]]).reshape(-1, n_kv, hd)
    T = len(x)
    for g in (1.0, 2.0 ** -20):
        bt = Batch([T], n_kv=n_kv, head_dim=hd, dtype=dtype, scale=g)
        k = (x * g).to(t)
        bt.write(bt.slots([T], [T]), k, -k)
        bt.assert_same_cache()
        bt.no_error()


def test_nan_infinity_and_the_far_ends():
    for dtype in ("f32", "bf16"):
        bt = Batch([5], n_kv=2, head_dim=32, dtype=dtype, scale=2.0 ** -60)
        x = bt.draw(5)
        x[0, 0, 3] = float("nan")
        x[1, 0, 3], x[1, 1, 20] = float("inf"), float("-inf")
        x[2] *= 2.0 ** -60
        x[3] *= 2.0 ** 60
        x[4, 0, 0], x[4, 0, 1] = float("nan"), float("inf")
        bt.write(bt.slots([5], [5]), x, x)
        bt.assert_same_cache()
        k, _ = gather(bt, [5], torch.float32)
        assert bool(k[0, 0, :16].isnan().all()) and bool(k[0, 0, 16:].isfinite().all())
        assert float(k[1, 0, 3]) == 2688 * 2.0 ** -60 and float(k[1, 1, 20]) == -2688 * 2.0 ** -60


@pytest.mark.parametrize("g", [2.0 ** -60, 2.0 ** -3, 2.0 ** 60])
def test_head_scales_over_their_range(g):
    bt = Batch([40], n_kv=3, head_dim=64, dtype="f32", scale=g)
    k, v = bt.draw(40) * g * 20, bt.draw(40) * g
    bt.write(bt.slots([40], [40]), k, v)
    bt.assert_same_cache()


@pytest.mark.parametrize("tokens,n_kv,head_dim", [(5000, 8, 64), (3000, 8, 128), (20000, 1, 16)])
def test_many_tokens(tokens, n_kv, head_dim):
    lens = [tokens // 4, tokens - tokens // 4]
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, seed=tokens)
    bt.fill()
    bt.assert_same_cache()
    k, v = gather(bt, lens)
    rows = [bt.rows(b, n) for b, n in enumerate(lens)]
    assert np.array_equal(f64(k), np.concatenate([r[0] for r in rows]))
    assert np.array_equal(f64(v), np.concatenate([r[1] for r in rows]))


def test_strided_rows_and_padding():
    """Rows of one projection's output; negative slots and slots past the pool."""
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([20], n_kv=4, head_dim=64)
    both = guarded_copy(torch.cat([bt.draw(20).flatten(1), bt.draw(20).flatten(1)], dim=1))
    k, v = both[:, :256].unflatten(1, (4, 64)), both[:, 256:].unflatten(1, (4, 64))
    slots = bt.slots([20], [20])
    slots[[2, 7]] = -1, -5
    slots[11], slots[12] = bt.nb * 16, 1 << 40
    pkv.kv_write_fp4(k, v, ints(slots, np.int64), *bt.cache, err=bt.err)
    assert int(bt.err.item()) == pkv.DEVERR["slot"]
    slots[[11, 12]] = -1
    bt.take(slots, f64(k), f64(v))
    bt.assert_same_cache()


def test_read_back_of_bad_batches():
    """Bad block ids, lengths and offsets give zeros and are reported."""
    import paged_kv_cache_write_gb300 as pkv
    lens = [40, 20]
    for what, bit in (("id", "block_id"), ("length", "length"), ("width", "table_width")):
        bt = Batch(lens, n_kv=2, head_dim=32)
        bt.fill()
        told = list(lens)
        cu = [0, 40, 60]
        if what == "id":
            bt.bt[0, 1] = bt.nb
            bt.bt[1, 0] = -1
        elif what == "length":
            told[1] = 5
        else:
            told[0], cu = 60, [0, 60, 80]
        n = cu[-1]
        k, v = pkv.kv_gather_fp4(*bt.cache, bt.bt, ints(told), ints(cu), n,
                                 k_out=guarded_empty((n, 2, 32), torch.float32),
                                 v_out=guarded_empty((n, 2, 32), torch.float32), err=bt.err)
        check_canaries()
        assert int(bt.err.item()) == pkv.DEVERR[bit]
        good = np.ones(n, dtype=bool)
        if what == "id":
            good[16:32] = good[40:56] = False
        elif what == "length":
            good[45:] = False
        else:
            good[48:60] = False
        assert not f64(k)[~good].any() and not f64(v)[~good].any()
        if what != "width":
            ref = np.concatenate([bt.rows(b, c)[0] for b, c in enumerate(lens)])
            assert np.array_equal(f64(k)[good], ref[good])


@pytest.mark.parametrize("n_kv,head_dim", [(1, 16), (3, 16), (5, 64), (8, 128)])
def test_a_shared_block_is_copied_then_written(n_kv, head_dim):
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([24, 24], n_kv=n_kv, head_dim=head_dim, spare=4)
    bt.fill()
    src, dst = int(bt.table[0, 1]), next(i for i in range(bt.nb) if i not in bt.table)
    pairs = ints([[src, dst]])
    pkv.copy_blocks(*(p.view(torch.bfloat16).view(bt.nb, 16, n_kv, head_dim // 4)
                      for p in (bt.d_kp, bt.d_vp)), pairs, err=bt.err)
    pkv.copy_blocks(*(g.view(bt.nb, -1).view(torch.float32).view(bt.nb, 1, 1, n_kv * head_dim // 4)
                      for g in (bt.d_kg, bt.d_vg)), pairs, err=bt.err)
    for x in (bt.kp, bt.vp, bt.kg, bt.vg):
        x[dst] = x[src]
    bt.no_error()
    bt.assert_same_cache()
    bt.table[1, :] = [bt.table[0, 0], dst]
    bt.write([dst * 16 + 8], bt.draw(1, 50.0), bt.draw(1, 50.0))
    bt.assert_same_cache()


@pytest.mark.parametrize("handle", [False, True])
def test_write_and_read_back_on_a_stream(handle):
    """Calls on a stream of their own, behind work that they have to wait for."""
    bt = Batch([30, 50], n_kv=4, head_dim=64, seed=5)
    t = 80
    k, v = (guarded_copy(bt.draw(t)) for _ in range(2))
    at, lens, cu = ints(bt.slots(bt.lens, bt.lens), np.int64), ints(bt.lens), ints([0, 30, 80])
    late_k, late_v = torch.zeros_like(k), torch.zeros_like(v)
    st = torch.cuda.Stream()
    where = st.cuda_stream if handle else st
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
        late_k.copy_(k)
        late_v.copy_(v)
    bt.pkv.kv_write_fp4(late_k, late_v, at, *bt.cache, err=bt.err, stream=where)
    x, y = bt.pkv.kv_gather_fp4(*bt.cache, bt.bt, lens, cu, t, err=bt.err, stream=where)
    st.synchronize()
    bt.take(bt.slots(bt.lens, bt.lens), f64(k), f64(v))
    bt.assert_same_cache()
    rows = [bt.rows(b, n) for b, n in enumerate(bt.lens)]
    assert np.array_equal(f64(x), np.concatenate([r[0] for r in rows]))
    assert np.array_equal(f64(y), np.concatenate([r[1] for r in rows]))
    bt.no_error()


def test_captured_write_and_read_back():
    bt = Batch([30, 50], n_kv=4, head_dim=64, seed=4)
    t = 80
    k, v = guarded_copy(bt.draw(t)), guarded_copy(bt.draw(t))
    slots = bt.slots(bt.lens, bt.lens)
    at, lens, cu = ints(slots, np.int64), ints(bt.lens), ints([0, 30, 80])
    outs = [guarded_empty((t, 4, 64), torch.bfloat16) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bt.pkv.kv_write_fp4(k, v, at, *bt.cache, err=bt.err)
        bt.pkv.kv_gather_fp4(*bt.cache, bt.bt, lens, cu, t, k_out=outs[0], v_out=outs[1], err=bt.err)
    for _ in range(3):
        x, y = bt.draw(t), bt.draw(t, 3.0)
        k.copy_(x)
        v.copy_(y)
        graph.replay()
        bt.take(slots, f64(x), f64(y))
        bt.assert_same_cache()
        rows = [bt.rows(b, n) for b, n in enumerate(bt.lens)]
        assert np.array_equal(f64(outs[0]), np.concatenate([r[0] for r in rows]))
        assert np.array_equal(f64(outs[1]), np.concatenate([r[1] for r in rows]))
    bt.no_error()
