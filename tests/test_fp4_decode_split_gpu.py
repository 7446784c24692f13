"""How a decode over the 4-bit cache splits its work: plans found in registers (to 256
sequences), in a CTA's shared memory or by a kernel of their own; clusters or a stream;
joins of few groups, captured and beside each other."""
import numpy as np
import pytest
import torch

from fp4_step import Batch, ints
from gpu_step import check_canaries, guarded_copy, guarded_empty

pytestmark = pytest.mark.gpu


def run(lens, heads, n_kv, head_dim, max_ctas, dtype="bf16", seed=0):
    lens = np.asarray(lens)
    bt = Batch(lens, n_kv=n_kv, head_dim=head_dim, dtype=dtype, seed=seed)
    bt.fill()
    q = bt.queries(len(lens), heads)
    out = bt.decode(q, max_ctas=max_ctas)
    again = bt.decode(q, max_ctas=max_ctas)
    bt.no_error()
    assert torch.equal(out, again)
    bt.check(out, q, range(len(lens)), lens - 1)
    return bt, q


def ragged(n, longest, seed):
    """Lengths to `longest`, a tenth of them zero, the ends among those."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, longest + 1, size=n)
    lens[rng.random(n) < 0.1] = 0
    lens[[0, -1]] = 0
    lens[n // 2] = longest
    return lens


# (n_kv 1 has groups of one head, whose lengths are read again; 8 keeps to 1,024 of them.
# With one head of 16 a CTA's ring has no room for more than some 830 sequences.)
@pytest.mark.parametrize("n,heads,n_kv,head_dim,dtype", [
    (256, 3, 1, 32, "bf16"), (257, 3, 1, 32, "bf16"), (600, 2, 1, 32, "f32"), (800, 2, 1, 16, "bf16"),
    (900, 2, 1, 16, "bf16"), (1024, 8, 8, 16, "bf16"), (1025, 8, 8, 16, "bf16"), (2048, 2, 2, 64, "bf16"),
    (2049, 2, 2, 64, "bf16"), (2100, 1, 1, 128, "f32"), (9000, 1, 1, 16, "bf16")])
@pytest.mark.parametrize("max_ctas", [7, 1000])
def test_streams_of_many_sequences(n, heads, n_kv, head_dim, dtype, max_ctas):
    run(ragged(n, 40, n), heads, n_kv, head_dim, max_ctas, dtype, seed=n)


@pytest.mark.parametrize("n,heads,n_kv,head_dim", [(257, 8, 8, 16), (300, 2, 1, 64), (1100, 4, 4, 32),
                                                   (2100, 8, 8, 16)])
def test_many_sequences_stream_by_themselves(n, heads, n_kv, head_dim):
    """One sequence is longer than a warp of a cluster may have it."""
    lens = ragged(n, 40, n)
    lens[n // 3] = 700
    run(lens, heads, n_kv, head_dim, 0, seed=n)


@pytest.mark.parametrize("heads,n_kv,head_dim,edge", [
    (8, 8, 128, 1280),   # ten blocks a warp of eight CTAs; one more and the call streams
    (8, 8, 64, 1664),    # thirteen
    (4, 2, 64, 2176)])   # seventeen
@pytest.mark.parametrize("more", [0, 1])
def test_one_sequence_at_the_border_of_clusters(heads, n_kv, head_dim, edge, more):
    run([edge + more], heads, n_kv, head_dim, 0)


@pytest.mark.parametrize("longest", [511, 512, 513])
def test_many_sequences_at_the_border_of_clusters(longest):
    """32 blocks a warp, whose ids fill a warp's lanes."""
    lens = ragged(310, 60, longest)
    lens[200] = longest
    run(lens, 16, 8, 16, 0, seed=longest)


@pytest.mark.parametrize("lens,heads,n_kv,head_dim", [([8000], 8, 2, 64), ([5000, 1, 0], 3, 1, 128),
                                                      ([6000, 17], 16, 8, 64)])
def test_few_long_sequences_captured_and_at_once(lens, heads, n_kv, head_dim):
    """Streams with a join of few groups: replayed with new queries, and two at a time."""
    import paged_kv_cache_write_gb300 as pkv
    bt, q1 = run(lens, heads, n_kv, head_dim, 0)
    q1, q2 = guarded_copy(q1), guarded_copy(bt.queries(len(lens), heads))
    sl, n = ints(lens), max(lens)
    need = pkv.decode_fp4_workspace_bytes(len(lens), heads, head_dim, n)
    ws = [guarded_empty((need,), torch.uint8) for _ in range(2)]

    def call(q, w, out, stream=None):
        pkv.paged_attention_decode_fp4(q, *bt.cache, bt.bt, sl, 0.125, n, out=out, workspace=w, err=bt.err,
                                       stream=stream)

    alone = [torch.empty_like(q1) for _ in range(2)]
    for q, o in zip((q1, q2), alone):
        call(q, ws[0], o)
        torch.cuda.synchronize()
    static, out = q1.clone(), torch.empty_like(q1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(static, ws[0], out)
        call(out, ws[0], static)  # reads what the join before it writes
        call(static, ws[0], out)
    for q in (q2, q1, q2):
        a, b = q.clone(), torch.empty_like(q)
        for x, y in ((a, b), (b, a), (a, b)):
            call(x, ws[1], y)
            torch.cuda.synchronize()
        static.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, b) and torch.equal(static, a)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q1) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, w, o in zip(streams, (q1, q2), ws, outs):
            call(q, w, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, alone))
    check_canaries()
    bt.no_error()


def test_two_planned_streams_at_once():
    """Batches whose plan is a kernel of its own, on two streams with a workspace each."""
    import paged_kv_cache_write_gb300 as pkv
    lens = ragged(2100, 40, 3)
    bt, q1 = run(lens, 4, 2, 16, 50)
    q1, q2 = guarded_copy(q1), guarded_copy(bt.queries(len(lens), 4))
    sl = ints(lens)
    need = pkv.decode_fp4_workspace_bytes(len(lens), 4, 16, 40, 50)
    ws = [guarded_empty((need,), torch.uint8) for _ in range(2)]
    outs = [guarded_empty(q1.shape, q1.dtype) for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]

    def call(i, out, stream=None):
        pkv.paged_attention_decode_fp4((q1, q2)[i], *bt.cache, bt.bt, sl, 0.25, 40, out=out, workspace=ws[i],
                                       max_ctas=50, err=bt.err, stream=stream)

    for i in range(2):
        call(i, outs[i])
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            call(i, outs[2 + i], streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    check_canaries()
    bt.no_error()


def test_infinity_in_a_query_shows():
    """Infinities of a query meet keys of both signs: its row is NaN, and the others are
    not touched, on every path of the decode and the prefill.  (Their last bits may be: the
    rows of a warp move their references together.)"""
    n = 300
    for hd, dtype in ((32, "bf16"), (64, "bf16"), (128, "bf16"), (64, "f32")):
        bt = Batch([n, n], n_kv=2, head_dim=hd, dtype=dtype, seed=hd)
        bt.fill()
        q = bt.queries(2, 4)
        bad = q.clone()
        bad[0, 1, 7], bad[1, 3, 2] = float("inf"), float("-inf")
        lens = [n, n]
        for call in (lambda x: bt.decode(x), lambda x: bt.decode(x, max_ctas=1),
                     lambda x: bt.decode(x, max_ctas=6), lambda x: bt.prefill(x, lens, [1, 1])):
            out = call(bad)
            bt.no_error()
            hit = torch.zeros(2, 4, dtype=torch.bool)
            hit[0, 1] = hit[1, 3] = True
            assert bool(out.cpu()[hit].isnan().all())
            ok = torch.where(hit[..., None], call(q).cpu(), out.cpu())
            bt.check(ok, q, range(2), [n - 1, n - 1])
