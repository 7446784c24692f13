"""Decode and prefill attention over the 4-bit cache against the float64
oracle on the cache's own values, with a tolerance derived from the kernels'
arithmetic (fp4_step.Batch.reference)."""
import numpy as np
import pytest
import torch

from fp4_step import Batch, f64, ints
from gpu_step import check_canaries, guarded_copy, guarded_empty

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[8000], [5000, 1, 0], [3000, 17, 16, 1100]])
@pytest.mark.parametrize("heads,n_kv,head_dim", [(8, 2, 64), (3, 1, 128), (16, 1, 16), (5, 5, 32)])
def test_decode_few_long_sequences(heads, n_kv, head_dim, lens, dtype):
    """Groups that many CTAs share."""
    _decode_case(heads, n_kv, head_dim, dtype, lens, 0, seed=heads)


@pytest.mark.parametrize("seqs,longest,heads,n_kv,head_dim,dtype", [
    (40, 1500, 16, 8, 64, "bf16"), (40, 1500, 8, 8, 128, "bf16"), (20, 2000, 16, 8, 64, "f32"),
    (280, 500, 8, 8, 16, "bf16"), (330, 500, 8, 8, 16, "f32"), (9, 1900, 12, 1, 64, "bf16")])
def test_decode_many_blocks_a_warp(seqs, longest, heads, n_kv, head_dim, dtype):
    """Whole sequences to a CTA or a cluster, with more blocks to a warp than it holds at once."""
    lens = np.random.default_rng(seqs).integers(0, longest + 1, size=seqs)
    lens[3] = longest
    _decode_case(heads, n_kv, head_dim, dtype, lens, 0, seed=seqs)


@pytest.mark.parametrize("lens", [[16, 5], [16, 0, 900], [0, 1]])
def test_decode_calls_in_a_row(lens):
    """Each call reads what the call before it wrote, where few groups, or none, are
    shared by CTAs though the longest length allowed would have them shared."""
    import paged_kv_cache_write_gb300 as pkv
    longest = 8192
    bt = Batch(lens, n_kv=2, head_dim=64, seed=4)
    bt.fill()
    sl = guarded_copy(torch.from_numpy(bt.lens))
    table = torch.zeros((len(lens), longest // 16), dtype=torch.int32, device="cuda")
    table[:, :bt.bt.shape[1]] = bt.bt
    ws = guarded_empty((pkv.decode_fp4_workspace_bytes(len(lens), 8, 64, longest),), torch.uint8)
    n = 24
    first = guarded_copy(bt.queries(len(lens), 8))

    def chain(wait):
        x = [first] + [torch.full_like(first, 3.0) for _ in range(n)]
        torch.cuda.synchronize()
        for i in range(n):
            pkv.paged_attention_decode_fp4(x[i], *bt.cache, table, sl, 0.125, longest,
                                           out=x[i + 1], workspace=ws, err=bt.err)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return torch.stack(x)

    apart = chain(True)
    bt.check(apart[1], first, range(len(lens)), bt.lens - 1)
    for _ in range(5):
        assert torch.equal(chain(False), apart)
    bt.no_error()


def test_decode_groups_far_apart():
    """Groups and heads whose scales differ as far as they can: nothing overflows or
    vanishes."""
    lens = [64, 200]
    for dtype in ("bf16", "f32"):
        for g in (2.0 ** -60, 1.0, 2.0 ** 30):
            bt = Batch(lens, n_kv=2, head_dim=64, dtype=dtype, seed=3, scale=g)
            t = sum(lens)
            k, v = bt.draw(t, 0.2).float() * g, bt.draw(t).float() * g
            v *= torch.exp2(torch.randint(-9, 8, (t, 2, 4), generator=bt.g).float()).repeat_interleave(16, -1)
            bt.write(bt.slots(lens, lens), k.to(bt.dtype), v.to(bt.dtype))
            q = (bt.queries(2, 8).float() / g).to(bt.dtype)
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
    for garbage, seed_blocks in (((0x77, 0x7F), 0), ((0, 0), 1), ((0xFF, 0xFE), 2)):
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
        bt.write(bt.slots([n, n], [n, n]), k, v)
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
            out = pkv.paged_attention_decode_fp4(guarded_copy(q), *bt.cache, bt.bt, sl, 0.125, 40,
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
    need = pkv.decode_fp4_workspace_bytes(3, 8, 64, n, max_ctas)
    ws = [guarded_empty((need,), torch.uint8) for _ in range(2)]

    def call(q, w, out, stream=None):
        return pkv.paged_attention_decode_fp4(q, *bt.cache, bt.bt, sl, 0.125, n, out=out,
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


@pytest.mark.parametrize("n_kv,head_dim", [(1, 64), (2, 128), (2, 32)])
def test_f32_sums_over_long_sequences(n_kv, head_dim):
    """Outputs of fp32 calls do not drift with the length.  The sums over 256 blocks are rounded
    at each (a random walk of sqrt(256 / 3) steps of 2^-24: 0.6e-6) and the scores, of a few
    units, are good to some 0.3e-6; sums that are cut off instead would be 256 x 2^-25 = 7.6e-6
    too small."""
    n, c = 4096, 24
    bt = Batch([n], n_kv=n_kv, head_dim=head_dim, dtype="f32", seed=1, scale=2.0 ** -6)
    k, v = bt.draw(n, 0.5), 1.0 + 0.25 * torch.randn(n, n_kv, head_dim, generator=bt.g)
    bt.write(bt.slots([n], [n]), k, v.float())
    q = bt.queries(c, 2 * n_kv, mag=0.2)
    outs = [(bt.prefill(q, [n], [c]), range(n - c, n))]
    for ctas in (0, 1, 7):
        outs.append((bt.decode(q[-1:], max_ctas=ctas), [n - 1]))
    bt.no_error()
    for out, lasts in outs:
        for i, last in enumerate(lasts):
            ref, _ = bt.reference(f64(q[i - len(lasts)]), 0, last)
            off = np.linalg.norm(f64(out[i]) - ref) / np.linalg.norm(ref)
            assert off <= 1.5e-6, (off, i, len(lasts))


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
def test_prefill_groups_far_apart(head_dim, dtype):
    for g in (2.0 ** -60, 2.0 ** 30):
        bt = Batch([300], n_kv=1, head_dim=head_dim, dtype=dtype, seed=6, scale=g)
        k, v = bt.draw(300, 0.2).float() * g, bt.draw(300).float() * g
        v *= torch.exp2(torch.randint(-9, 8, (300, 1, head_dim // 16), generator=bt.g).float()
                        ).repeat_interleave(16, -1)
        bt.write(bt.slots([300], [300]), k.to(bt.dtype), v.to(bt.dtype))
        q = (bt.queries(300, 2).float() / g).to(bt.dtype)
        out = bt.prefill(q, [300], [300])
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
        bt.write(bt.slots([n], [n]), k, v)
        q = bt.queries(n, 4, mag=0.3)
        out = bt.prefill(q, [n], [n])
        bt.no_error()
        assert bool(out[:at].isfinite().all())
        seen = out[at:]
        if what == "k":
            assert bool(seen.isnan().all())
        else:
            assert bool(seen[..., :16].isnan().all()) and bool(seen[..., 16:].isfinite().all())
        clean = Batch([n], n_kv=1, head_dim=head_dim, dtype=dtype, seed=4)
        ck, cv = clean.draw(n), clean.draw(n)
        (ck if what == "k" else cv)[at, 0, 3] = 0.0
        clean.write(clean.slots([n], [n]), ck, cv)
        clean.check(out[:at], q[:at], [0] * at, range(at), held=4)


@pytest.mark.parametrize("seqs,heads,n_kv,head_dim", [(300, 8, 8, 64), (150, 16, 8, 128),
                                                      (700, 6, 3, 64), (600, 4, 2, 128)])
def test_prefill_many_chunks(seqs, heads, n_kv, head_dim):
    """Far more work items than the GPU takes at once, in both orders of them (more than 512
    sequences have the natural one), with NaNs that some queries see: every sequence's rows are
    those of a call for it alone, and as the oracle has them."""
    import paged_kv_cache_write_gb300 as pkv
    rng = np.random.default_rng(seqs)
    lens = rng.integers(1, 150, size=seqs)
    new = np.minimum(lens, rng.integers(0, 150, size=seqs))
    lens[5], new[5] = 700, 600
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, seed=seqs)
    t = int(lens.sum())
    k, v = bt.draw(t), bt.draw(t)
    end = np.cumsum(lens)
    # every third sequence: a NaN value at a position that part of its queries see
    at = np.where((np.arange(seqs) % 3 == 0) & (new > 1), lens - new // 2, lens)
    for b in np.flatnonzero(at < lens):
        v[end[b] - lens[b] + at[b], b % n_kv, 17] = float("nan")
    bt.write(bt.slots(lens, lens), k, v)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = bt.queries(int(cu[-1]), heads)
    out = bt.prefill(q, lens, new)
    bt.no_error()
    rep = heads // n_kv
    nan = out.isnan()
    for b in range(seqs):
        rows, first = nan[cu[b]:cu[b + 1]].cpu(), int(at[b] - (lens[b] - new[b]))
        hit = torch.zeros_like(rows)
        hit[first:, (b % n_kv) * rep:(b % n_kv + 1) * rep, 16:32] = bool(at[b] < lens[b])
        assert torch.equal(rows, hit), b
    dq = guarded_copy(q)
    for b in list(range(0, seqs, 37)) + [5]:
        c = int(new[b])
        if c == 0:
            continue
        alone = pkv.paged_attention_prefill_fp4(
            dq[cu[b]:cu[b + 1]], ints([0, c]), *bt.cache, bt.bt[b:b + 1], ints(lens[b:b + 1]),
            1.0 / np.sqrt(head_dim), c, int(lens[b]), err=bt.err)
        torch.cuda.synchronize()
        assert torch.equal(alone.view(torch.int16), out[cu[b]:cu[b + 1]].view(torch.int16)), b
    some = [(b, i) for b in range(1, seqs, 11) if at[b] == lens[b]
            for i in range(0, int(new[b]), 23)]
    at_rows = [cu[b] + i for b, i in some]
    bt.check(out[at_rows], q[at_rows], [b for b, _ in some],
             [int(lens[b] - new[b] + i) for b, i in some], held=4)


@pytest.mark.parametrize("head_dim,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32")])
def test_prefill_captured_and_at_once(head_dim, dtype):
    """Two calls that run side by side (streams given as objects and as handles), each with more
    work than the GPU takes at once, and a captured one over new queries, give what each gives
    alone."""
    import paged_kv_cache_write_gb300 as pkv
    rng = np.random.default_rng(9)
    lens = rng.integers(1, 200, size=90)
    bt = Batch(lens, n_kv=4, head_dim=head_dim, dtype=dtype, seed=9)
    bt.fill()
    t = int(lens.sum())
    qs = [guarded_copy(bt.queries(t, 8)) for _ in range(2)]
    cu, sl = ints(np.concatenate([[0], np.cumsum(lens)])), ints(lens)

    def call(q, out, stream=None):
        return pkv.paged_attention_prefill_fp4(q, cu, *bt.cache, bt.bt, sl, 0.125, int(lens.max()),
                                               int(lens.max()), out=out, err=bt.err, stream=stream)

    alone = [call(q, torch.empty_like(q)).clone() for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.full_like(q, 7.0) for q in qs]
    torch.cuda.synchronize()
    for i in range(12):
        for s, q, o in zip(streams, qs, outs):
            call(q, o, stream=s if i % 2 else s.cuda_stream)
    torch.cuda.synchronize()
    for o, ref in zip(outs, alone):
        assert torch.equal(o, ref)
    static, out = qs[0].clone(), torch.empty_like(qs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(static, out)
        call(static, out)
    for k in (1, 0, 1):
        static.copy_(qs[k])
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, alone[k])
    bt.no_error()


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
        bt.write(bt.slots(have, new), bt.draw(t), bt.draw(t))
        q = bt.queries(t, heads)
        out = bt.prefill(q, have, new)
        which = [b for b, c in enumerate(new) for _ in range(c)]
        bt.check(out, q, which, [n - c + i for n, c in zip(have, new) for i in range(c)],
                 held=4)
    for s in range(1, steps + 1):
        have = prompt + s
        bt.write(bt.slots(have, [1] * 4), bt.draw(4, 1.0 + s % 3), bt.draw(4, 1.0 + s % 4))
        q = bt.queries(4, heads)
        out = bt.decode(q, lens=have)
        bt.check(out, q, range(4), have - 1)
    bt.no_error()
    bt.assert_same_cache()


def test_step_in_one_graph():
    """Norm, rotation and write, decode and the next layer's, captured together:
    early-launching kernels wait for the cache and the queries that the step writes."""
    import paged_kv_cache_write_gb300 as pkv
    from test_norm_rope_gpu import Step
    lens = np.array([700, 18, 1100, 33])
    layers = [Batch(lens, n_kv=2, head_dim=64, seed=s) for s in (1, 2, 3)]
    for b in layers:
        t = int((lens - 1).sum())
        b.write(b.slots(lens - 1, lens - 1), b.draw(t), b.draw(t))
    sl = ints(lens)
    steps = [Step(4, 8, 2, 64, 64, "bf16", seed=s) for s in (4, 5, 6)]
    slots = [ints(b.slots(lens, [1] * 4), np.int64) for b in layers]
    qs = [guarded_empty(s.q.shape, s.dtype) for s in steps]
    outs = [guarded_empty(q.shape, q.dtype) for q in qs]
    ws = guarded_empty((pkv.decode_fp4_workspace_bytes(4, 8, 64, 1100),), torch.uint8)

    def run(between=lambda: None):
        for b, s, at, q, o in zip(layers, steps, slots, qs, outs):
            pkv.qk_norm_rope_write_fp4(s.q, s.k, s.v, *s.args, at, *b.cache, **s.kw_args, q_out=q, err=b.err)
            between()
            pkv.paged_attention_decode_fp4(q, *b.cache, b.bt, sl, 0.125, 1100, out=o, workspace=ws, err=b.err)
            between()

    run(torch.cuda.synchronize)
    alone = [x.clone() for x in outs + qs]
    caches = [[x.clone() for x in b.cache] for b in layers]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for again in range(4):
        for b in layers:  # the step's tokens are gone
            for x in b.cache[2:4]:
                x.view(torch.uint8).view(b.nb, 2, 16, 4)[[int(v) // 16 for v in b.slots(lens, [1] * 4)], :,
                                                         [int(v) % 16 for v in b.slots(lens, [1] * 4)]] = 0
        for x in outs + qs:
            x.zero_()
        graph.replay() if again < 3 else run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs + qs, alone))
        for b, old in zip(layers, caches):
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(b.cache, old))
    check_canaries()
    for b, s, q, o in zip(layers, steps, qs, outs):
        k = paged_keys(s)
        b.take(b.slots(lens, [1] * 4), k, s.v.float().cpu().numpy().astype(np.float64))
        b.assert_same_cache()
        b.check(o, q.cpu(), range(4), lens - 1)
        b.no_error()


def paged_keys(s):
    """The keys of a Step as they are rounded before they are quantised."""
    import paged_kv_cache_write_gb300 as pkv
    _, k = pkv.qk_norm_rope(s.q, s.k, *s.args, **s.kw_args)
    return k.float().cpu().numpy().astype(np.float64)


# ---------------------------------------------------------- bad device data

# (head_dim, type, sequences): tcgen05 with an ordered and with a plain grid (more than
# 512 sequences), warp-level products
PATHS = [(64, "bf16", 3), (128, "bf16", 3), (64, "bf16", 600), (128, "bf16", 600), (16, "bf16", 3),
         (32, "bf16", 3), (64, "f32", 3), (128, "f32", 3)]


def chunks(head_dim, dtype, n):
    """n sequences of 40 tokens and the last 6 of each as a chunk."""
    bt = Batch([40] * n, n_kv=1, head_dim=head_dim, dtype=dtype, seed=n)
    bt.fill()
    return bt, bt.queries(6 * n, 2), [40] * n, [6] * n


@pytest.mark.parametrize("head_dim,dtype,n", PATHS)
def test_any_block_id_out_of_range_is_reported(head_dim, dtype, n):
    """-1, the usual filler of a table, is a bad id where it stands for a block that the
    sequence holds; it is read as zeros like any other."""
    import paged_kv_cache_write_gb300 as pkv
    bt, q, lens, new = chunks(head_dim, dtype, n)
    good = bt.prefill(q, lens, new)
    bt.no_error()
    seen = []
    for bad in (-7, -1, bt.nb, -2 ** 31, 2 ** 31 - 1):
        bt.bt[1, 1] = bad
        out = bt.prefill(q, lens, new)
        torch.cuda.synchronize()
        assert int(bt.err.item()) == pkv.DEVERR["block_id"], bad
        assert torch.equal(out[:6], good[:6]) and torch.equal(out[12:], good[12:])
        seen.append(out[6:12].clone())
        bt.err.zero_()
    assert all(torch.equal(x, seen[0]) for x in seen) and not torch.equal(seen[0], good[6:12])
    # zeros: as a block of zero codes and scales
    bt.bt.copy_(torch.from_numpy(bt.table))
    for x in bt.cache[:4]:
        x.view(torch.uint8)[int(bt.table[1, 1])] = 0
    assert torch.equal(bt.prefill(q, lens, new)[6:12], seen[0])


@pytest.mark.parametrize("head_dim,dtype,n", PATHS)
def test_filler_behind_a_sequences_blocks_is_not_reported(head_dim, dtype, n):
    bt, q, lens, new = chunks(head_dim, dtype, n)
    good = bt.prefill(q, lens, new)
    dec = bt.decode(q[:n].contiguous())
    wide = np.full((n, 9), -1, dtype=np.int32)
    wide[:, :3] = bt.table
    bt.bt = guarded_copy(torch.from_numpy(wide))
    assert torch.equal(bt.prefill(q, lens, new), good)
    assert torch.equal(bt.decode(q[:n].contiguous()), dec)
    bt.no_error()


# offsets of 3 chunks over 18 query rows that disagree with the rows, with each other or
# with the largest chunk (6); the chunks that hold all the same
@pytest.mark.parametrize("cu,good", [([0, 6, 12, 16], (0, 1)),           # stop short of the rows
                                     ([0, 6, 12, 30], (0, 1)),           # go past them
                                     ([12, 6, 12, 18], (1, 2)),          # go back
                                     ([0, 6, 15, 18], (0, 2)),           # a chunk longer than max_q_len
                                     ([0, 2 ** 31 - 1, 12, 18], (2,)),
                                     ([0, 1 << 20, 1 << 20, 1 << 20], ()),
                                     ([-6, 0, 12, 18], (2,))])
@pytest.mark.parametrize("head_dim,dtype,n", PATHS)
def test_offsets_that_disagree_are_reported(head_dim, dtype, n, cu, good):
    """Rows that belong to no chunk are left as they were."""
    import paged_kv_cache_write_gb300 as pkv
    bt, q, lens, new = chunks(head_dim, dtype, n)
    table = bt.bt.flip(0).contiguous()
    cu = ints([cu[0]] * (n - 3) + cu)
    out, want = (guarded_empty((18, 2, head_dim), bt.dtype) for _ in range(2))
    out.fill_(7.0)
    q3 = guarded_copy(q[:18])
    s = 1.0 / np.sqrt(head_dim)
    pkv.paged_attention_prefill_fp4(q3, cu, *bt.cache, table, ints(lens), s, 6, 40, out=out, err=bt.err)
    torch.cuda.synchronize()
    assert int(bt.err.item()) == pkv.DEVERR["length"]
    bt.err.zero_()
    pkv.paged_attention_prefill_fp4(q3, ints([0] * (n - 3) + [0, 6, 12, 18]), *bt.cache, table, ints(lens), s,
                                    6, 40, out=want, err=bt.err)
    bt.no_error()
    at = cu[-4:].tolist()
    owned = torch.zeros(18, dtype=torch.bool, device="cuda")
    for i in range(3):
        lo, hi = max(0, at[i]), min(18, at[i + 1])
        owned[lo:hi] = True
        if i in good and (lo, hi) == (6 * i, 6 * i + 6):
            assert torch.equal(out[lo:hi], want[lo:hi]), i
    assert bool((out[~owned] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("head_dim", [32, 64, 128])
@pytest.mark.parametrize("step", [13, 40])
def test_scores_that_grow_from_tile_to_tile(head_dim, dtype, step):
    """Keys in runs of 64 whose scores are some `step` log2 units above the run before,
    for every other query head; the others' stay within a few units (rows that keep
    their reference beside rows that move it).  Repeated calls give the same bits."""
    n, heads = 640, 4
    bt = Batch([n], n_kv=1, head_dim=head_dim, dtype=dtype, seed=step, scale=2.0 ** -4)
    k = torch.randn(n, 1, head_dim, generator=bt.g) * 0.05
    run = torch.arange(n) // 64
    k[:, 0, 0] = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 8.0, 12.0])[run]
    k[:, 0, 1] = torch.rand(n, generator=bt.g)
    bt.write(bt.slots([n], [n]), k.to(bt.dtype), bt.draw(n))
    q = torch.randn(n, heads, head_dim, generator=bt.g) * 0.05
    q[..., :2] = 0
    q[:, ::2, 0] = step * np.log(2) * np.sqrt(head_dim)
    q[:, 1::2, 1] = np.log(2) * np.sqrt(head_dim)
    q = q.to(bt.dtype)
    outs = [bt.prefill(q, [n], [n]) for _ in range(12)]
    bt.no_error()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    bt.check(outs[0], q, [0] * n, range(n), held=4)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("n,head_dim,dtype", [(5, 64, "bf16"), (5, 32, "bf16"), (5, 128, "f32"),
                                              (700, 64, "bf16"), (40, 128, "bf16")])
def test_lengths_offsets_and_tables_written_by_the_kernel_before(n, head_dim, dtype, captured):
    """Each call follows the kernels that write its lengths, offsets and table without a
    wait; between calls they hold zeros."""
    import paged_kv_cache_write_gb300 as pkv
    rng = np.random.default_rng(n)
    most = 40 if n > 100 else 300
    lens = rng.integers(3, most, size=n)
    lens[::2] = most
    bt = Batch(lens, n_kv=2, head_dim=head_dim, dtype=dtype, seed=n)
    bt.fill()
    real = [ints(x) for x in (lens, np.arange(n + 1), np.concatenate([[0], np.cumsum(lens)]), bt.table)]
    sl, cu, full, table = held = [torch.zeros_like(x) for x in real]
    total = int(lens.sum())
    q = guarded_copy(bt.queries(n, 8))
    ws = guarded_empty((pkv.decode_fp4_workspace_bytes(n, 8, head_dim, most),), torch.uint8)
    outs = [guarded_empty((m, h, head_dim), bt.dtype) for m, h in ((n, 8), (n, 8), (total, 2), (total, 2))]
    s = 1.0 / np.sqrt(head_dim)

    def step(between=lambda: None):
        def written(last):
            for x in held:
                torch.mul(x, 0, out=x)
            for x, y in sorted(zip(held, real), key=lambda xy: xy[0] is last):
                torch.add(y, 0, out=x)
            between()

        for last in (sl, table):
            written(last)
            pkv.paged_attention_decode_fp4(q, *bt.cache, table, sl, s, most, out=outs[0], workspace=ws,
                                           err=bt.err)
            between()
        for last in (sl, cu, table):
            written(last)
            pkv.paged_attention_prefill_fp4(q, cu, *bt.cache, table, sl, s, 1, most, out=outs[1], err=bt.err)
            between()
        for last in (sl, full, table):
            written(last)
            pkv.kv_gather_fp4(*bt.cache, table, sl, full, total, k_out=outs[2], v_out=outs[3], err=bt.err)
            between()

    step(torch.cuda.synchronize)
    ref = [x.clone() for x in outs]
    bt.no_error()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
    for _ in range(8):
        for x in outs:
            x.zero_()
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, ref))
    bt.no_error()


def test_a_pool_past_4_gib():
    """Blocks whose codes lie past 2^32 bytes, in every reading and writing entry."""
    import paged_kv_cache_write_gb300 as pkv
    n_kv, hd = 32, 128
    nb = (1 << 32) // (n_kv * 16 * hd // 2) + 40
    bt = Batch([70, 33], n_kv=n_kv, head_dim=hd, seed=1)
    bt.fill()
    big = [torch.empty((nb, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in bt.cache[:4]]
    far = torch.from_numpy(bt.table).cuda() + (nb - bt.nb)
    slots = ints(bt.slots(bt.lens, bt.lens) + (nb - bt.nb) * 16, np.int64)
    k, v = pkv.kv_gather_fp4(*bt.cache, bt.bt, ints(bt.lens), ints([0, 70, 103]), 103)
    pkv.kv_write_fp4(k, v, slots, *big, *bt.cache[4:], err=bt.err)
    k2, v2 = pkv.kv_gather_fp4(*big, *bt.cache[4:], far, ints(bt.lens), ints([0, 70, 103]), 103, err=bt.err)
    ref = Batch([70, 33], n_kv=n_kv, head_dim=hd, seed=1)
    pkv.kv_write_fp4(k, v, ints(bt.slots(bt.lens, bt.lens), np.int64), *ref.cache)
    k3, v3 = pkv.kv_gather_fp4(*ref.cache, bt.bt, ints(bt.lens), ints([0, 70, 103]), 103)
    assert torch.equal(k2, k3) and torch.equal(v2, v3)
    q = guarded_copy(bt.queries(2, 64))
    for ctas in (0, 3):
        a = pkv.paged_attention_decode_fp4(q, *big, *bt.cache[4:], far, ints(bt.lens), 0.1, 70, max_ctas=ctas)
        b = pkv.paged_attention_decode_fp4(q, *ref.cache, bt.bt, ints(bt.lens), 0.1, 70, max_ctas=ctas)
        assert torch.equal(a, b)
    cu = ints([0, 1, 2])
    for x in (q, q.float()):
        a = pkv.paged_attention_prefill_fp4(x, cu, *big, *bt.cache[4:], far, ints(bt.lens), 0.1, 1, 70)
        b = pkv.paged_attention_prefill_fp4(x, cu, *ref.cache, bt.bt, ints(bt.lens), 0.1, 1, 70)
        assert torch.equal(a, b)
    bt.no_error()
