"""Decode and prefill attention over the 8-bit cache against the float64
oracle on the cache's own values, with a tolerance derived from the kernels'
arithmetic (fp8_step.Batch.reference)."""
import numpy as np
import pytest
import torch

from fp8_step import Batch, f64
from gpu_step import guarded_copy, guarded_empty

pytestmark = pytest.mark.gpu

HEADS = [(4, 2), (8, 4), (9, 3), (1, 1), (16, 1), (12, 1), (26, 2), (32, 8), (11, 11), (40, 8)]


def _decode_case(heads, n_kv, head_dim, dtype, lens, max_ctas, seed=0, mag=1.0):
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, dtype=dtype, seed=seed)
    bt.fill(mag)
    q = bt.queries(len(lens), heads)
    out = bt.decode(q, max_ctas=max_ctas)
    bt.no_error()
    bt.check(out, q, range(len(lens)), [n - 1 for n in lens])
    return bt, q, out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("head_dim", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,n_kv", HEADS)
def test_decode_heads(heads, n_kv, head_dim, dtype):
    """Every head grouping, cluster path (max_ctas 0) and stream path."""
    lens = [1, 15, 16, 17, 0, 100, 33]
    for ctas in (0, 1, 5):
        _decode_case(heads, n_kv, head_dim, dtype, lens, ctas, seed=heads)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("max_ctas", [0, 1, 3, 16, 1000])
def test_decode_long_and_ragged(max_ctas, dtype):
    """Sequences past the cluster path's 64 blocks, split over many CTAs; more
    than 32 and 64 blocks in one CTA's range (scales are fetched 32 at a time)."""
    _decode_case(8, 2, 64, dtype, [1500, 1, 0, 2047, 513, 1024, 70], max_ctas, seed=7)


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [16], [1024], [1025], [31] * 40])
def test_decode_small_batches(lens):
    for hd in (64, 128):
        _decode_case(8, 8, hd, "bf16", lens, 0, seed=len(lens))


def test_decode_many_sequences():
    """Batches planned in every CTA and by the plan kernel (over 2,048)."""
    rng = np.random.default_rng(1)
    for n in (600, 2600):
        lens = rng.integers(0, 30, size=n)
        bt = Batch(lens, n_kv=1, head_dim=32, seed=n)
        bt.fill()
        q = bt.queries(n, 3)
        out = bt.decode(q)
        bt.no_error()
        bt.check(out, q, range(n), lens - 1)


def test_decode_scales_far_apart():
    """Blocks whose K and V scales differ by many powers of two: weights go
    where the values are large, and nothing overflows or vanishes."""
    lens = [64, 200]
    for dtype in ("bf16", "f32"):
        bt = Batch(lens, n_kv=2, head_dim=64, dtype=dtype, seed=3)
        t = sum(lens)
        k, v = bt.draw(t, 0.2), bt.draw(t).float()
        v *= torch.exp2(torch.randint(-30, 30, (t // 16 + 1, 1, 1), generator=bt.g).float()
                        ).repeat_interleave(16, 0)[:t]
        bt.write(lens, lens, k, v.to(bt.dtype))
        q = bt.queries(2, 8)
        for ctas in (0, 1, 4):
            out = bt.decode(q, max_ctas=ctas)
            bt.no_error()
            bt.check(out, q, range(2), [n - 1 for n in lens])


def test_decode_large_and_small_queries():
    """Queries far outside f16's range, rows of zeros."""
    bt = Batch([50, 60, 40], n_kv=2, head_dim=64, seed=5)
    bt.fill(2.0 ** -20)
    q = bt.queries(3, 4).float()
    q[0] *= 2.0 ** 20
    q[1] *= 2.0 ** -100
    q[2, 1] = 0
    q = q.to(torch.bfloat16)
    for ctas in (0, 2):
        out = bt.decode(q, max_ctas=ctas)
        bt.check(out, q, range(3), [49, 59, 39])


def test_decode_ignores_what_is_not_its_own():
    """The same outputs whatever bytes lie past the lengths and in other
    blocks, and under any physical placement."""
    lens = [5, 30, 17, 900]
    outs = []
    for garbage, seed_blocks in ((0x7F, 0), (0x00, 1), (0x7E, 2)):
        bt = Batch(lens, n_kv=2, head_dim=128, garbage=garbage, seed=11)
        perm = np.random.default_rng(seed_blocks).permutation(bt.nb)
        bt.table = perm[bt.table].astype(np.int32)
        bt.bt.copy_(torch.from_numpy(bt.table))
        bt.fill()
        q = bt.queries(4, 8)
        outs.append([bt.decode(q, max_ctas=c) for c in (0, 1, 7)])
        pre = bt.prefill(q, lens, [1, 1, 1, 1])
        outs[-1].append(pre)
        bt.no_error()
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def test_decode_nan_in_a_visible_key_shows():
    """NaN and infinity that a query sees make its output NaN, on every path,
    and only its own."""
    for ctas, n in ((0, 40), (1, 40), (6, 400)):
        bt = Batch([n, n], n_kv=2, head_dim=64, seed=2)
        k, v = bt.draw(2 * n), bt.draw(2 * n)
        k[n // 2, 0, 5] = float("nan")  # sequence 0, KV head 0
        bt.write([n, n], [n, n], k, v)
        q = bt.queries(2, 4)
        out = bt.decode(q, max_ctas=ctas)
        torch.cuda.synchronize()
        assert bool(out[0, :2].isnan().all())
        assert bool(out[0, 2:].isfinite().all()) and bool(out[1].isfinite().all())


def test_decode_bad_device_data():
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([40, 20], n_kv=2, head_dim=64)
    bt.fill()
    q = bt.queries(2, 4)
    good = bt.decode(q)
    bt.bt[0, 1] = bt.nb  # read as zeros
    for ctas in (0, 1):
        bt.err.zero_()
        out = bt.decode(q, max_ctas=ctas)
        torch.cuda.synchronize()
        assert int(bt.err.item()) == pkv.DEVERR["block_id"] and bool(out.isfinite().all())
        assert torch.equal(out[1], bt.decode(q, max_ctas=ctas)[1])
    bt.bt.copy_(torch.from_numpy(bt.table))
    for lens, bit in (([-3, 20], "length"), ([40, 2 ** 31 - 1], "length")):
        for ctas in (0, 1):
            bt.err.zero_()
            sl = guarded_copy(torch.tensor(lens, dtype=torch.int32))
            out = pkv.paged_attention_decode_fp8(guarded_copy(q), *bt.cache, bt.bt, sl, 0.125, 40,
                                                 max_ctas=ctas, err=bt.err)
            torch.cuda.synchronize()
            assert int(bt.err.item()) == pkv.DEVERR[bit]
            if lens[0] < 0:
                assert not out[0].any()
    assert good.shape == q.shape


@pytest.mark.parametrize("max_ctas,n", [(0, 60), (0, 1500), (9, 300)])
def test_decode_captured_and_on_streams(max_ctas, n):
    """A captured call replays with new inputs; calls on two streams with a
    workspace each give what they give alone."""
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([n, 3, n // 2], n_kv=2, head_dim=64, seed=8)
    bt.fill()
    q1, q2 = (guarded_copy(bt.queries(3, 8)) for _ in range(2))
    sl = guarded_copy(torch.from_numpy(bt.lens))
    need = pkv.decode_fp8_workspace_bytes(3, 8, 64, n, max_ctas)
    ws = [guarded_empty((need,), torch.uint8) for _ in range(2)]

    def call(q, w, out, stream=None):
        return pkv.paged_attention_decode_fp8(q, *bt.cache, bt.bt, sl, 0.125, n, out=out,
                                              workspace=w, max_ctas=max_ctas, err=bt.err, stream=stream)

    alone = [call(q, ws[0], torch.empty_like(q)).clone() for q in (q1, q2)]
    torch.cuda.synchronize()
    static, out = q1.clone(), torch.empty_like(q1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(static, ws[0], out)
    for q, ref in ((q2, alone[1]), (q1, alone[0]), (q2, alone[1])):
        static.copy_(q)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q1) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, w, o in zip(streams, (q1, q2), ws, outs):
            call(q, w, o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])
    bt.no_error()


# ----------------------------------------------------------------- prefill

def _prefill_case(heads, n_kv, head_dim, dtype, lens, new, seed=0):
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, dtype=dtype, seed=seed)
    bt.fill()
    q = bt.queries(sum(new), heads)
    out = bt.prefill(q, lens, new)
    bt.no_error()
    which = [b for b, c in enumerate(new) for _ in range(c)]
    last = [n - c + i for n, c in zip(lens, new) for i in range(c)]
    bt.check(out, q, which, last, held=4)
    return bt, q, out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("head_dim", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,n_kv", HEADS)
def test_prefill_heads(heads, n_kv, head_dim, dtype):
    _prefill_case(heads, n_kv, head_dim, dtype, [1, 16, 40, 65, 9, 130], [1, 16, 24, 1, 9, 37],
                  seed=heads)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,new", [([300], [300]), ([700], [5]), ([257, 129], [129, 128]),
                                      ([530, 3, 128], [270, 0, 128])])
def test_prefill_lengths(lens, new, dtype):
    """Several query and key tiles, chunks that end on and beside tile limits,
    a sequence without a query."""
    for heads, n_kv, hd in ((6, 2, 64), (4, 1, 128)):
        _prefill_case(heads, n_kv, hd, dtype, lens, new, seed=len(lens))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("head_dim", [32, 64, 128])
def test_prefill_scales_far_apart(head_dim, dtype):
    lens = [300]
    bt = Batch(lens, n_kv=1, head_dim=head_dim, dtype=dtype, seed=6)
    k, v = bt.draw(300, 0.2), bt.draw(300).float()
    v *= torch.exp2(torch.randint(-20, 20, (19, 1, 1), generator=bt.g).float()).repeat_interleave(16, 0)[:300]
    bt.write(lens, lens, k, v.to(bt.dtype))
    q = bt.queries(300, 2)
    out = bt.prefill(q, lens, [300])
    bt.no_error()
    bt.check(out, q, [0] * 300, range(300), held=4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("head_dim", [32, 64, 128])
def test_prefill_hidden_nan_stays_hidden(head_dim, dtype):
    """NaN in a key or a value reaches exactly the queries that see it."""
    n, at = 150, 77
    for what in ("k", "v"):
        bt = Batch([n], n_kv=1, head_dim=head_dim, dtype=dtype, seed=4)
        k, v = bt.draw(n), bt.draw(n)
        (k if what == "k" else v)[at, 0, 3] = float("nan")
        bt.write([n], [n], k, v)
        q = bt.queries(n, 4, mag=0.3)
        out = bt.prefill(q, [n], [n])
        bt.no_error()
        assert bool(out[:at].isfinite().all())
        seen = out[at:]
        if what == "k":
            assert bool(seen.isnan().all())
        else:
            assert bool(seen[..., 3].isnan().all())
            keep = [d for d in range(head_dim) if d != 3]
            assert bool(seen[..., keep].isfinite().all())
        clean = Batch([n], n_kv=1, head_dim=head_dim, dtype=dtype, seed=4)
        ck, cv = clean.draw(n), clean.draw(n)
        (ck if what == "k" else cv)[at, 0, 3] = 0.0
        clean.write([n], [n], ck, cv)
        clean.check(out[:at], q[:at], [0] * at, range(at), held=4)


def test_prefill_bad_device_data():
    import paged_kv_cache_write_gb300 as pkv
    for hd, dtype in ((32, torch.bfloat16), (64, torch.bfloat16), (128, torch.float32)):
        bt = Batch([40, 20], n_kv=1, head_dim=hd, dtype={torch.bfloat16: "bf16"}.get(dtype, "f32"))
        bt.fill()
        q = bt.queries(12, 2)
        bt.bt[0, 1] = -7
        out = bt.prefill(q, [40, 20], [6, 6])
        torch.cuda.synchronize()
        assert int(bt.err.item()) == pkv.DEVERR["block_id"] and bool(out.isfinite().all())
        bt.bt.copy_(torch.from_numpy(bt.table))
        for lens, bit in (([3, 20], "length"), ([-1, 20], "length")):
            bt.err.zero_()
            bt.prefill(q, lens, [6, 6])
            torch.cuda.synchronize()
            assert int(bt.err.item()) == pkv.DEVERR[bit]


# --------------------------------------------------------- as they are used

@pytest.mark.parametrize("heads,n_kv,head_dim,dtype", [(8, 4, 16, "f32"), (9, 3, 64, "bf16"),
                                                       (16, 2, 128, "bf16")])
def test_prompts_then_decode_steps(heads, n_kv, head_dim, dtype):
    """A serving loop: prompts written and prefilled in two chunks, then
    decode steps that each append a token; every output of every step against
    the oracle on the cache as it then is, and the cache itself at the end."""
    prompt, steps = np.array([1, 37, 16, 90]), 18
    bt = Batch(prompt + steps, n_kv=n_kv, head_dim=head_dim, dtype=dtype, seed=1)
    first = prompt // 2
    for have, new in ((first, first), (prompt, prompt - first)):
        t = int(new.sum())
        bt.write(have, new, bt.draw(t), bt.draw(t))
        q = bt.queries(t, heads)
        out = bt.prefill(q, have, new)
        which = [b for b, c in enumerate(new) for _ in range(c)]
        bt.check(out, q, which, [n - c + i for n, c in zip(have, new) for i in range(c)],
                 held=4)
    for s in range(1, steps + 1):
        have = prompt + s
        bt.write(have, [1] * 4, bt.draw(4, 1.0 + s % 3), bt.draw(4, 1.0 + s % 4))
        q = bt.queries(4, heads)
        out = bt.decode(q, lens=have)
        bt.check(out, q, range(4), have - 1)
    bt.no_error()
    bt.assert_same_cache()


def test_step_in_one_graph():
    """Write, decode and the next layer's write and decode captured together:
    early-launching kernels wait for the cache that the step writes."""
    lens = np.array([700, 18, 1100, 33])
    layers = [Batch(lens, n_kv=2, head_dim=64, seed=s) for s in (1, 2, 3)]
    for b in layers:
        t = int((lens - 1).sum())
        b.write(lens - 1, lens - 1, b.draw(t), b.draw(t))
    import paged_kv_cache_write_gb300 as pkv
    sl = guarded_copy(torch.from_numpy(lens.astype(np.int32)))
    cu = guarded_copy(torch.arange(5, dtype=torch.int32))
    new = [tuple(b.draw(4, 2.0) for _ in range(2)) for b in layers]
    dev = [tuple(guarded_copy(x) for x in kv) for kv in new]
    qs = [guarded_copy(b.queries(4, 8)) for b in layers]
    outs = [guarded_empty(q.shape, q.dtype) for q in qs]
    ws = guarded_empty((pkv.decode_fp8_workspace_bytes(4, 8, 64, 1100),), torch.uint8)

    def step():
        for b, (k, v), q, o in zip(layers, dev, qs, outs):
            pkv.kv_write_fp8(k, v, b.bt, sl, cu, *b.cache, err=b.err)
            pkv.paged_attention_decode_fp8(q, *b.cache, b.bt, sl, 0.125, 1100, out=o, workspace=ws,
                                           err=b.err)

    before = [[x.clone() for x in b.cache] for b in layers]
    step()
    torch.cuda.synchronize()
    eager = [o.clone() for o in outs]
    for b, old in zip(layers, before):
        for x, y in zip(b.cache, old):
            x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for b, kv, q, o, e in zip(layers, new, qs, outs, eager):
        assert torch.equal(o, e)
        b.write(lens, [1] * 4, *kv)  # the oracle's cache takes the step (the GPU's again, unchanged)
        b.assert_same_cache()
        b.check(o, q.cpu(), range(4), lens - 1)
        b.no_error()
