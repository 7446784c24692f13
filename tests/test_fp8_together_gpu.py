"""The 8-bit cache's entries as a serving loop calls them: captured and
replayed in one chain, on several streams over one cache, with padded and very
large batches.  Calls that do the same are compared bit for bit."""
import numpy as np
import pytest
import torch

from fp8_step import Batch, f64
from gpu_step import guarded_copy, guarded_empty

pytestmark = pytest.mark.gpu


def ints(x):
    return guarded_copy(torch.as_tensor(np.asarray(x, dtype=np.int32)))


class Chain:
    """Write of one token a sequence, read-back, decode, prefill of a chunk of
    one, over the sequences `rows` of a cache; inputs and outputs kept."""

    def __init__(self, bt, rows, heads, most, have):
        import paged_kv_cache_write_gb300 as pkv
        self.pkv, self.bt, n = pkv, bt, len(rows)
        self.table = guarded_copy(bt.bt[torch.as_tensor(rows).cuda()].contiguous())
        self.sl = ints(have)
        self.one = ints(np.arange(n + 1))
        self.full = ints(np.concatenate([[0], np.cumsum(have)]))
        self.total, self.most = int(np.sum(have)), most
        self.k, self.v = (guarded_empty((n, bt.n_kv, bt.hd), bt.dtype) for _ in range(2))
        self.q = guarded_copy(bt.queries(n, heads))
        self.dec, self.pre = (guarded_empty(self.q.shape, bt.dtype) for _ in range(2))
        self.kb, self.vb = (guarded_empty((self.total, bt.n_kv, bt.hd), bt.dtype) for _ in range(2))
        self.ws = guarded_empty((pkv.decode_fp8_workspace_bytes(n, heads, bt.hd, most),), torch.uint8)

    def put(self, seed):
        """New tokens, larger from step to step, so that scales grow."""
        g = torch.Generator().manual_seed(seed)
        for t in (self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=g) * 1.3 ** seed)

    def run(self, between=lambda: None):
        pkv, bt, c = self.pkv, self.bt, self.bt.cache
        s = 1.0 / np.sqrt(bt.hd)
        pkv.kv_write_fp8(self.k, self.v, self.table, self.sl, self.one, *c, err=bt.err)
        between()
        pkv.kv_gather_fp8(*c, self.table, self.sl, self.full, self.total, k_out=self.kb,
                          v_out=self.vb, err=bt.err)
        between()
        pkv.paged_attention_decode_fp8(self.q, *c, self.table, self.sl, s, self.most, out=self.dec,
                                       workspace=self.ws, err=bt.err)
        between()
        pkv.paged_attention_prefill_fp8(self.q, self.one, *c, self.table, self.sl, s, 1, self.most,
                                        out=self.pre, err=bt.err)
        between()
        # the same token again, as the next layer would: nothing may change
        pkv.kv_write_fp8(self.k, self.v, self.table, self.sl, self.one, *c, err=bt.err)
        between()

    def results(self):
        return [x.clone() for x in (self.kb, self.vb, self.dec, self.pre)]


def caches(bt):
    return [x.view(torch.uint8).clone() if x.dtype.itemsize == 1 else x.clone() for x in bt.cache]


def restore(bt, state):
    for x, y in zip(bt.cache, state):
        (x.view(torch.uint8) if x.dtype.itemsize == 1 else x).copy_(y)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("n_kv,head_dim,dtype,n", [(8, 64, "bf16", 40), (4, 16, "f32", 9),
                                                   (2, 128, "bf16", 300)])
def test_chain_in_a_graph(n_kv, head_dim, dtype, n):
    """The captured chain, whose kernels start while the preceding one ends,
    leaves what its calls leave when each is waited for."""
    lens = np.random.default_rng(n).integers(2, 330, size=n)
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, dtype=dtype, seed=n)
    t = int((lens - 1).sum())
    bt.write(lens - 1, lens - 1, bt.draw(t), bt.draw(t))
    ch = Chain(bt, np.arange(n), 4 * n_kv, int(lens.max()), lens)
    ch.put(0)
    before = caches(bt)
    expect = []
    for step in range(12):
        ch.put(step)
        torch.cuda.synchronize()
        ch.run(torch.cuda.synchronize)
        expect.append(ch.results() + caches(bt))
    restore(bt, before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ch.run()
    for step in range(12):
        ch.put(step)
        for x in (ch.kb, ch.vb, ch.dec, ch.pre):
            x.fill_(7.0)
        graph.replay()
        assert same(ch.results() + caches(bt), expect[step]), step
    bt.no_error()


def test_chains_on_two_streams_over_one_cache():
    """Two streams, each with its own half of a cache's sequences."""
    lens = np.random.default_rng(5).integers(2, 300, size=60)
    bt = Batch(lens, n_kv=2, head_dim=64, seed=5)
    t = int((lens - 1).sum())
    bt.write(lens - 1, lens - 1, bt.draw(t), bt.draw(t))
    halves = [Chain(bt, r, 8, int(lens.max()), lens[r]) for r in (np.arange(0, 60, 2), np.arange(1, 60, 2))]
    before = caches(bt)
    expect = []
    for step in range(10):
        for ch in halves:
            ch.put(step)
            ch.run(torch.cuda.synchronize)
        expect.append([x for ch in halves for x in ch.results()] + caches(bt))
    restore(bt, before)
    streams = [torch.cuda.Stream() for _ in halves]
    for step in range(10):
        for ch in halves:
            ch.put(step)
        torch.cuda.synchronize()
        for s, ch in zip(streams, halves):
            with torch.cuda.stream(s):
                ch.run()
        torch.cuda.synchronize()
        assert same([x for ch in halves for x in ch.results()] + caches(bt), expect[step]), step
    bt.no_error()


@pytest.mark.parametrize("raw", [False, True])
def test_stream_argument(raw):
    """A stream given by object or address; what the call allocates for itself
    belongs to that stream."""
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([100, 17], n_kv=2, head_dim=64)
    bt.fill()
    ref = {}
    sl, cu = ints(bt.lens), ints([0, 100, 117])
    # sequence 1 holds what it reads back as (the scales of values that were
    # rounded down may be smaller), so that the writes below change nothing
    k, v = pkv.kv_gather_fp8(*bt.cache, bt.bt, sl, cu, 117, dtype=torch.float32)
    pkv.kv_write_fp8(k[-17:].contiguous(), v[-17:].contiguous(), bt.bt[1:], sl[1:], ints([0, 17]),
                     *bt.cache, err=bt.err)
    q, one = guarded_copy(bt.queries(2, 8)), ints([0, 1, 2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for name, s in (("current", None), ("side", side.cuda_stream if raw else side), ("legacy", 0)):
        k, v = pkv.kv_gather_fp8(*bt.cache, bt.bt, sl, cu, 117, dtype=torch.float32, stream=s)
        assert k.dtype == torch.float32
        d = pkv.paged_attention_decode_fp8(q, *bt.cache, bt.bt, sl, 0.125, stream=s)
        p = pkv.paged_attention_prefill_fp8(q, one, *bt.cache, bt.bt, sl, 0.125, stream=s)
        pkv.kv_write_fp8(k[-17:].contiguous(), v[-17:].contiguous(), bt.bt[1:], sl[1:],
                         ints([0, 17]), *bt.cache, err=bt.err,
                         stream=s)
        torch.cuda.synchronize()
        ref[name] = [k, v, d, p] + caches(bt)
    assert same(ref["current"], ref["side"]) and same(ref["current"], ref["legacy"])
    bt.no_error()


@pytest.mark.parametrize("head_dim,dtype", [(64, "bf16"), (32, "f32"), (128, "bf16")])
def test_padded_batch(head_dim, dtype):
    """Rows of length 0 whose tables name nothing, before, between and behind
    the sequences: they get zeros (decode) and change no other row."""
    import paged_kv_cache_write_gb300 as pkv
    lens = np.array([130, 1, 60])
    a = Batch(lens, n_kv=2, head_dim=head_dim, dtype=dtype, seed=3)
    b = Batch(lens, n_kv=2, head_dim=head_dim, dtype=dtype, seed=3)
    k, v, q = a.draw(191), a.draw(191), a.queries(3, 8)
    qp = a.queries(191, 8)
    at = [1, 2, 5]
    wide = np.full((8, b.table.shape[1]), -1, dtype=np.int32)
    wide[at] = b.table
    wl = np.zeros(8, dtype=np.int64)
    wl[at] = lens
    wq = torch.full((8, 8, head_dim), float("nan"), dtype=q.dtype)
    wq[at] = q
    a.write(lens, lens, k, v)
    b.table, b.bt = wide, guarded_copy(torch.from_numpy(wide))
    b.write(wl, wl, k, v)
    assert same(caches(a), caches(b))
    da, db = a.decode(q), b.decode(wq, lens=wl)
    assert torch.equal(da, db[torch.tensor(at)]) and not bool(db[torch.tensor([0, 3, 4, 6, 7])].any())
    assert torch.equal(a.prefill(qp, lens, lens), b.prefill(qp, wl, wl))
    full = [ints(np.concatenate([[0], np.cumsum(x)])) for x in (lens, wl)]
    ga = pkv.kv_gather_fp8(*a.cache, a.bt, ints(lens), full[0], 191, err=a.err)
    gb = pkv.kv_gather_fp8(*b.cache, b.bt, ints(wl), full[1], 191, err=b.err)
    assert same(ga, gb)
    a.no_error()
    b.no_error()


@pytest.mark.parametrize("head_dim,dtype", [(64, "bf16"), (32, "f32")])
def test_batches_past_the_grids_extents(head_dim, dtype):
    """70,000 sequences of one token.  The only weight is (nearly) 1, so an
    output is off by its weight's rounding (2^-11 for bf16, less for fp32) before
    it is rounded itself: the value, a number of 4 bits, exactly for bf16."""
    import paged_kv_cache_write_gb300 as pkv
    n = 70_000
    bt = Batch(np.ones(n), n_kv=1, head_dim=head_dim, dtype=dtype, spare=0)
    k, v, q = (torch.randn(n, 1, head_dim, device="cuda").to(bt.dtype) for _ in range(3))
    sl, cu = ints(np.ones(n)), ints(np.arange(n + 1))
    pkv.kv_write_fp8(k, v, bt.bt, sl, cu, *bt.cache, err=bt.err)
    kb, vb = pkv.kv_gather_fp8(*bt.cache, bt.bt, sl, cu, n, dtype=bt.dtype, err=bt.err)
    assert bool(((kb.float() - k.float()).abs() <= k.float().abs() * 2 ** -4 + 2 ** -10).all())
    dec = pkv.paged_attention_decode_fp8(q, *bt.cache, bt.bt, sl, 0.1, 1, err=bt.err)
    pre = pkv.paged_attention_prefill_fp8(q, cu, *bt.cache, bt.bt, sl, 0.1, 1, 1, err=bt.err)
    for out in (dec, pre):
        if dtype == "bf16":
            assert torch.equal(out, vb)
        else:
            assert bool(((out - vb).abs() <= vb.abs() * 2 ** -20).all())
    bt.no_error()


@pytest.mark.parametrize("n", [1500, 3000])
def test_decode_many_sequences_some_long(n):
    """More sequences than have their lengths kept on chip, planned in every
    CTA and by the plan kernel, some over many blocks."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 20, size=n)
    lens[rng.integers(0, n, size=5)] = rng.integers(1100, 1500, size=5)
    bt = Batch(lens, n_kv=2, head_dim=16, seed=n)
    bt.fill()
    q = bt.queries(n, 4)
    out = bt.decode(q)
    bt.no_error()
    bt.check(out, q, range(n), lens - 1)


@pytest.mark.parametrize("head_dim", [64, 128])
def test_prefill_more_sequences_than_are_ordered(head_dim):
    lens = np.random.default_rng(2).integers(1, 40, size=600)
    new = np.minimum(lens, np.random.default_rng(3).integers(0, 9, size=600))
    bt = Batch(lens, n_kv=1, head_dim=head_dim, seed=2)
    bt.fill()
    q = bt.queries(int(new.sum()), 4)
    out = bt.prefill(q, lens, new)
    bt.no_error()
    which = [b for b, c in enumerate(new) for _ in range(c)]
    bt.check(out, q, which, [n - c + i for n, c in zip(lens, new) for i in range(c)], held=4)


def test_offsets_that_go_back_are_reported():
    """cu_new_lens that decrease: such a range has no tokens to read."""
    import paged_kv_cache_write_gb300 as pkv
    bt = Batch([20, 7, 18, 4], n_kv=2, head_dim=32)
    k = guarded_copy(bt.draw(4))
    for cu in ([0, 3, 1, 2, 4], [0, 4, 0, 4, 4], [4, 3, 2, 1, 0], [0, 2 ** 31 - 1, -2 ** 31, 1, 4],
               [-7, -3, 1, 2, 4]):
        bt.err.zero_()
        pkv.kv_write_fp8(k, k, bt.bt, ints(bt.lens), ints(cu), *bt.cache, err=bt.err)
        torch.cuda.synchronize()
        assert int(bt.err.item()) in (0, pkv.DEVERR["length"]), cu
        if cu[1:] != [4, 0, 4, 4]:  # (there each token still has one range around it)
            assert int(bt.err.item()) == pkv.DEVERR["length"], cu


def test_prefill_longer_than_it_was_told():
    import paged_kv_cache_write_gb300 as pkv
    for hd, dtype in ((64, "bf16"), (32, "bf16"), (128, "f32")):
        bt = Batch([40, 20], n_kv=1, head_dim=hd, dtype=dtype)
        bt.fill()
        q = guarded_copy(bt.queries(4, 2))
        out = pkv.paged_attention_prefill_fp8(q, ints([0, 2, 4]), *bt.cache, bt.bt, ints([40, 20]),
                                              0.1, 2, 30, err=bt.err)
        torch.cuda.synchronize()
        assert int(bt.err.item()) == pkv.DEVERR["length"]
        assert bool(out[2:].isfinite().all())
        bt.err.zero_()
        good = pkv.paged_attention_prefill_fp8(q, ints([0, 2, 4]), *bt.cache, bt.bt, ints([40, 20]),
                                               0.1, 2, 40, err=bt.err)
        assert np.array_equal(f64(good[2:]), f64(out[2:]))
        bt.no_error()


def test_calls_from_two_threads():
    """Two host threads, each with shapes of its own that the same kernels are
    launched with in different sizes."""
    import threading
    shapes = [(8, 8, 64), (9, 3, 64), (6, 2, 64), (5, 1, 64)]
    batches = [Batch([1500, 700, 30], n_kv=kv, head_dim=hd, seed=i)
               for i, (_, kv, hd) in enumerate(shapes)]
    qs, alone = [], []
    for bt, (heads, _, _) in zip(batches, shapes):
        bt.fill()
        qs.append(bt.queries(3, heads))
        alone.append(bt.decode(qs[-1]))
    torch.cuda.synchronize()
    bad = []

    def work(mine):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(150):
                    for j in mine:
                        out = batches[j].pkv.paged_attention_decode_fp8(
                            d_q[j], *batches[j].cache, batches[j].bt, lens[j],
                            1.0 / np.sqrt(batches[j].hd), 1500, err=batches[j].err)
                    if i % 50 == 49:
                        torch.cuda.current_stream().synchronize()
                        if not torch.equal(out, alone[mine[-1]]):
                            bad.append((mine, i))
        except Exception as e:  # noqa: BLE001 (reported below)
            bad.append(e)

    d_q = [guarded_copy(q) for q in qs]
    lens = [ints([1500, 700, 30]) for _ in shapes]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(m,)) for m in ([0, 1], [2, 3])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad
    for bt in batches:
        bt.no_error()
