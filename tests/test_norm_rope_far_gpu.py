"""Norm and rotation of rows at the ends of the types' ranges, of infinities and NaN, both
rotations into a 4-bit cache, and the write before a planned decode."""
import numpy as np
import pytest
import torch

from fp4_step import Batch, f64, ints
from gpu_step import check_canaries, guarded_copy, guarded_empty
from oracle import paged_fp4
from test_norm_rope_gpu import Step, rows_out

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -126, 2.0 ** -101, 2.0 ** -99, 1e-5])
@pytest.mark.parametrize("hd,rot,interleaved", [(16, 16, False), (64, 32, True), (80, 80, False),
                                                (256, 256, False)])
def test_rows_of_every_size(hd, rot, interleaved, eps, dtype):
    """Rows of one warp whose squares vanish, are as usual and overflow."""
    s = Step(5, 12, 4, hd, rot, dtype, eps=eps, interleaved=interleaved, seed=hd)
    far = 2.0 ** torch.tensor([0, -60, -120, 60, 90, 0, -52, -48, -70, 55, -110, 20], dtype=torch.float64)
    for x in (s.q, s.k):
        x.copy_((x.double() * far[:x.shape[1], None].cuda()).to(s.dtype))
    s.x = [f64(t) for t in (s.q, s.k)]
    q, k = rows_out(s)
    s.check(q, 0)
    s.check(k, 1)
    assert int(s.err.item()) == 0


def expect(s, i, got):
    """Not-a-numbers and infinities where the formula has them; other rows as ever."""
    w = f64((s.qw, s.kw)[i]) if s.qw is not None else None
    with np.errstate(invalid="ignore", over="ignore"):
        ref = paged_fp4.norm_rope(s.x[i], w, s.eps, s.cs.numpy(), s.positions, s.interleaved)
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isposinf(got), np.isposinf(ref)) and np.array_equal(np.isneginf(got), np.isneginf(ref))
    rows = np.isfinite(s.x[i]).all(axis=-1)
    fine = s.x[i].copy()
    fine[~rows] = 1.0
    clean = Step.__new__(Step)
    clean.__dict__.update(s.__dict__)
    clean.x = [fine, fine]
    clean.check(torch.from_numpy(np.where(rows[..., None], got, 0.0)), i, rows) if rows.any() else None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["both", "none"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_and_nan(interleaved, norm, dtype):
    s = Step(6, 4, 2, 64, 32, dtype, norm, interleaved, seed=11)
    inf, nan = float("inf"), float("nan")
    s.q[0, 0, 3], s.q[1, 1, 20], s.q[2, 2, 40], s.q[3, 3, 63] = inf, -inf, nan, inf
    s.k[0, 1, 31], s.k[4, 0, 16], s.k[4, 0, 0] = nan, inf, -inf
    s.x = [f64(t) for t in (s.q, s.k)]
    q, k = rows_out(s)
    expect(s, 0, q)
    expect(s, 1, k)
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,n_kv,hd,rot", [(1, 8, 4, 16, 16), (70, 8, 2, 64, 64), (33, 4, 2, 64, 32),
                                                 (20, 10, 5, 96, 48), (40, 4, 2, 128, 128), (90, 6, 3, 256, 16)])
def test_both_rotations_into_a_4_bit_cache(T, heads, n_kv, hd, rot, interleaved, dtype):
    """Bit for bit the rows, then their write; and the oracle's codes of those rows."""
    import paged_kv_cache_write_gb300 as pkv
    s = Step(T, heads, n_kv, hd, rot, dtype, interleaved=interleaved, seed=T)
    a, b = (Batch([T], n_kv=n_kv, head_dim=hd, dtype=dtype, seed=2) for _ in range(2))
    slots = a.slots([T], [T])
    if T > 8:
        slots[3], slots[5] = -1, a.nb * 16
    q, k = rows_out(s)
    s.check(q, 0)
    s.check(k, 1)
    pkv.kv_write_fp4(k, s.v, ints(slots, np.int64), *a.cache, err=a.err)
    q2 = pkv.qk_norm_rope_write_fp4(s.q, s.k, s.v, *s.args, ints(slots, np.int64), *b.cache, **s.kw_args,
                                    err=b.err)
    check_canaries()
    assert torch.equal(q, q2)
    for x, y in zip(a.cache, b.cache):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert int(a.err.item()) == int(b.err.item()) == (pkv.DEVERR["slot"] if T > 8 else 0)
    slots[slots >= a.nb * 16] = -1
    a.take(slots, f64(k), f64(s.v))
    a.assert_same_cache()


def test_write_before_a_planned_decode():
    """A planned decode reads its first blocks before it waits for the kernel ahead of it,
    so the write of this step's keys and values must not let it in: layer after layer, in
    turn with other work of this library, captured and not."""
    import paged_kv_cache_write_gb300 as pkv
    lens = [5, 16, 33, 1, 47, 20, 8, 64] * 8
    n, heads, n_kv, hd, nb = len(lens), 16, 8, 64, 4 * 64
    g = torch.Generator().manual_seed(0)
    table = torch.randperm(nb, generator=g).int().view(n, 4)
    bt, sl = guarded_copy(table), ints(lens)
    slots = ints([int(table[b, (L - 1) // 16]) * 16 + (L - 1) % 16 for b, L in enumerate(lens)], np.int64)
    steps = [Step(n, heads, n_kv, hd, hd, "bf16", seed=i) for i in range(4)]
    fresh = [[torch.randn(nb, 16, n_kv, hd, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
             for _ in steps]
    pools = [[guarded_copy(x) for x in f] for f in fresh]
    four = Batch([64], n_kv=n_kv, head_dim=hd, seed=1)
    four_slots = ints(four.slots([64], [64]), np.int64)
    ws = guarded_empty((pkv.decode_workspace_bytes(n, heads, hd, 64),), torch.uint8)
    qs = [guarded_empty(s.q.shape, s.dtype) for s in steps]
    outs = [guarded_empty(s.q.shape, s.dtype) for s in steps]
    err = guarded_empty((1,), torch.int32)
    err.zero_()
    pkv.decode_plan(pools[0][0], sl, heads, 4, 64, workspace=ws, err=err)
    torch.cuda.synchronize()

    def run(between, mixed):
        for s, p, q, o in zip(steps, pools, qs, outs):
            pkv.qk_norm_rope_write(s.q, s.k, s.v, *s.args, slots, *p, **s.kw_args, q_out=q, err=err)
            between()
            if mixed:  # lets the next kernel in early, after it has waited itself
                pkv.kv_write_fp4(s.k, s.v, four_slots, *four.cache, err=err)
                between()
            pkv.paged_attention_decode_planned(q, *p, bt, sl, 0.125, 64, workspace=ws, out=o, err=err)
            between()

    def restore():
        for p, f in zip(pools, fresh):
            for x, y in zip(p, f):
                x.copy_(y)
        for x in qs + outs:
            x.zero_()

    run(torch.cuda.synchronize, False)
    alone = [x.clone() for x in outs + qs]
    plain = [pkv.paged_attention_decode(q, *p, bt, sl, 0.125, 64) for q, p in zip(qs, pools)]
    assert all(torch.equal(a, b) for a, b in zip(plain, outs))
    for mixed in (False, True):
        graph = torch.cuda.CUDAGraph()
        restore()
        torch.cuda.synchronize()
        unguarded = pkv.paged_attention_decode_planned.__wrapped__
        guarded, pkv.paged_attention_decode_planned = pkv.paged_attention_decode_planned, unguarded
        try:
            with torch.cuda.graph(graph):
                run(lambda: None, mixed)
            for again in range(6):
                restore()
                graph.replay() if again < 4 else run(lambda: None, mixed)
                torch.cuda.synchronize()
                assert all(torch.equal(x, y) for x, y in zip(outs + qs, alone))
        finally:
            pkv.paged_attention_decode_planned = guarded
    check_canaries()
    assert int(err.item()) == 0
