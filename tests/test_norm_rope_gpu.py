"""Norm and rotation of queries and keys, alone and with the write into a cache,
against the float64 oracle."""
import numpy as np
import pytest
import torch

from fp4_step import HALF, TYPES, Batch, f64, ints
from gpu_step import check_canaries, guarded_copy, guarded_empty
from oracle import paged_fp4

pytestmark = pytest.mark.gpu


def table(positions, rot, base=10000.0):
    half = rot // 2
    angle = np.arange(positions)[:, None] * base ** (-np.arange(half) / half)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], axis=1)).float()


def bound(x, weight, eps, cos_sin, positions, interleaved, dtype):
    """How far a result may be from the oracle's.  A sum of head_dim squares in fp32 is
    off relatively by at most head_dim 2^-24, its root by half that and 1 / sqrt by two
    units more (2^-22); the other products and sums, six of them, by 2^-24 each of
    |z cos| + |z' sin|; then half a step of the result."""
    z = np.abs(x)
    if weight is not None:
        z = z / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.abs(weight)
    both = np.abs(cos_sin.astype(np.float64))
    half = both.shape[-1] // 2
    far = z.copy()
    row = both[positions][:, None, :]
    c, s = row[..., :half], row[..., half:]
    lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
              else (slice(0, half), slice(half, 2 * half)))
    far[..., lo] = z[..., lo] * c + z[..., hi] * s
    far[..., hi] = z[..., hi] * c + z[..., lo] * s
    rel = (x.shape[-1] / 2 + 6) * 2.0 ** -24 + 2.0 ** -22
    ref = paged_fp4.norm_rope(x, weight, eps, cos_sin, positions, interleaved)
    return ref, HALF[dtype] * np.abs(ref) + (1 + HALF[dtype]) * rel * far + 1e-37


class Step:
    """A projection's output of T tokens with some gap between them."""

    def __init__(self, T, heads, n_kv, hd, rot, dtype, norm="both", interleaved=False, seed=0, pad=0,
                 eps=1e-5):
        g = torch.Generator().manual_seed(seed)
        self.T, self.heads, self.n_kv, self.hd = T, heads, n_kv, hd
        self.dtype = TYPES[dtype]
        width = (heads + 2 * n_kv) * hd + pad
        self.qkv = guarded_copy((3 * torch.randn(T, width, generator=g)).to(self.dtype))
        at = [0, heads * hd, (heads + n_kv) * hd, (heads + 2 * n_kv) * hd]
        self.q, self.k, self.v = (self.qkv[:, a:b].unflatten(1, (-1, hd)) for a, b in zip(at, at[1:]))
        self.x = [f64(t) for t in (self.q, self.k)]
        w = [(1 + 0.3 * torch.randn(hd, generator=g)).to(self.dtype) for _ in range(2)]
        self.qw, self.kw = (None if norm in ("none", other) else guarded_copy(t)
                            for t, other in zip(w, ("k", "q")))
        self.eps, self.interleaved = eps, interleaved
        self.cs = table(500, rot)
        self.positions = np.random.default_rng(seed).integers(0, 500, T)
        self.args = guarded_copy(self.cs), ints(self.positions)
        self.kw_args = dict(q_weight=self.qw, k_weight=self.kw, eps=eps, interleaved=interleaved)
        self.err = guarded_empty((1,), torch.int32)
        self.err.zero_()

    def check(self, got, i, rows=None):
        w = (self.qw, self.kw)[i]
        ref, tol = bound(self.x[i], None if w is None else f64(w), self.eps, self.cs.numpy(),
                         self.positions, self.interleaved, self.dtype)
        far = np.abs(f64(got) - ref) / tol
        far = far if rows is None else far[rows]
        assert far.size == 0 or far.max() <= 1, far.max()


def rows_out(s, **kw):
    import paged_kv_cache_write_gb300 as pkv
    q = guarded_empty(s.q.shape, s.dtype)
    k = guarded_empty(s.k.shape, s.dtype)
    pkv.qk_norm_rope(s.q, s.k, *s.args, **s.kw_args, q_out=q, k_out=k, err=s.err, **kw)
    check_canaries()
    return q, k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", ["both", "none", "q", "k"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hd,rot", [(16, 16), (32, 32), (32, 16), (48, 32), (64, 64), (80, 80), (96, 48),
                                    (128, 128), (128, 32), (208, 112), (256, 256), (256, 16)])
def test_rows(hd, rot, interleaved, norm, dtype):
    for T, heads, n_kv in ((1, 1, 1), (5, 9, 3), (3, 4, 1)):
        s = Step(T, heads, n_kv, hd, rot, dtype, norm, interleaved, seed=hd + rot, pad=16 * (T % 3))
        q, k = rows_out(s)
        s.check(q, 0)
        s.check(k, 1)
        assert int(s.err.item()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,heads,n_kv,hd", [(700, 64, 8, 128), (9000, 3, 1, 32), (2500, 32, 8, 64)])
def test_many_tokens(T, heads, n_kv, hd, dtype):
    """Warps that go through several rows of a token."""
    s = Step(T, heads, n_kv, hd, hd, dtype, seed=T)
    q, k = rows_out(s)
    s.check(q, 0)
    s.check(k, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [16, 64, 96, 128])
def test_in_place(hd, dtype):
    """Results over the rows that they come from, in the projection's output."""
    import paged_kv_cache_write_gb300 as pkv
    s = Step(37, 8, 4, hd, hd, dtype, seed=hd)
    q, k = rows_out(s)
    before = s.v.clone()
    pkv.qk_norm_rope(s.q, s.k, *s.args, **s.kw_args, q_out=s.q, k_out=s.k, err=s.err)
    check_canaries()
    assert torch.equal(s.q, q) and torch.equal(s.k, k) and torch.equal(s.v, before)


def test_rows_of_zeros_and_far_values():
    """Rows of zeros stay zeros (eps); rows of 2^60 and 2^-60 keep their size without a
    norm and lose it with one."""
    for norm in ("both", "none"):
        s = Step(4, 2, 1, 64, 64, "f32", norm, seed=1, eps=0.0 if norm == "none" else 1e-5)
        s.q[0] = 0
        s.k[0] = 0
        s.q[1] *= 2.0 ** 60
        s.q[2] *= 2.0 ** -60
        s.x = [f64(t) for t in (s.q, s.k)]
        q, k = rows_out(s)
        s.check(q, 0)
        s.check(k, 1)
        assert not q[0].any() and not k[0].any()


def test_bad_positions_give_zeros_and_store_nothing():
    import paged_kv_cache_write_gb300 as pkv
    s = Step(6, 4, 2, 32, 32, "bf16", seed=3)
    bad = s.positions.copy()
    bad[1], bad[4] = 500, -1
    s.args = s.args[0], ints(bad)
    q, k = rows_out(s)
    assert int(s.err.item()) == pkv.DEVERR["length"]
    good = [0, 2, 3, 5]
    s.check(q, 0, good)
    s.check(k, 1, good)
    assert not q[[1, 4]].any() and not k[[1, 4]].any()
    pools = [guarded_copy(torch.full((2, 16, 2, 32), 7.0).to(s.dtype)) for _ in range(2)]
    slots = np.array([0, 3, 31, 17, 8, 9])
    pkv.qk_norm_rope_write(s.q, s.k, s.v, *s.args, ints(slots, np.int64), *pools, **s.kw_args, err=s.err)
    for p in pools:
        rows = p.view(32, 2, 32)
        assert bool((rows[[3, 8]] == 7).all()) and not bool((rows[[0, 31, 17, 9]] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,heads,n_kv,hd,bs", [(1, 8, 4, 16, 16), (64, 32, 8, 64, 16), (300, 9, 3, 64, 4),
                                                (33, 10, 5, 80, 1), (40, 4, 2, 256, 16)])
def test_write_equals_rows_then_kv_write(T, heads, n_kv, hd, bs, dtype):
    """Bit for bit; padded tokens and slots past the pool store nothing."""
    import paged_kv_cache_write_gb300 as pkv
    s = Step(T, heads, n_kv, hd, hd // 32 * 16 or 16, dtype, seed=T, interleaved=T % 2 == 0)
    nb = T // bs + 3
    slots = np.random.default_rng(T).permutation(nb * bs)[:T]
    if T > 8:
        slots[3], slots[5] = -1, nb * bs
    q, k = rows_out(s)
    g = torch.Generator().manual_seed(1)
    fresh = [torch.randn(nb, bs, n_kv, hd, generator=g).to(s.dtype) for _ in range(2)]
    ref, got = ([guarded_copy(x) for x in fresh] for _ in range(2))
    at = ints(slots, np.int64)
    pkv.kv_write(k, guarded_copy(s.v), at, *ref, err=s.err)
    err2 = guarded_empty((1,), torch.int32)
    err2.zero_()
    q2 = pkv.qk_norm_rope_write(s.q, s.k, s.v, *s.args, at, *got, **s.kw_args, err=err2)
    check_canaries()
    assert torch.equal(q, q2) and all(torch.equal(a, b) for a, b in zip(ref, got))
    assert int(err2.item()) == int(s.err.item()) == (pkv.DEVERR["slot"] if T > 8 else 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,heads,n_kv,hd", [(1, 8, 4, 16), (70, 32, 8, 64), (33, 10, 5, 96), (40, 4, 2, 128),
                                             (700, 6, 3, 256)])
def test_write_fp4_equals_rows_then_kv_write_fp4(T, heads, n_kv, hd, dtype):
    import paged_kv_cache_write_gb300 as pkv
    s = Step(T, heads, n_kv, hd, hd // 32 * 16 or 16, dtype, seed=T, norm="k")
    a, b = (Batch([T], n_kv=n_kv, head_dim=hd, dtype=dtype, seed=2) for _ in range(2))
    slots = a.slots([T], [T])
    if T > 8:
        slots[3], slots[5] = -1, a.nb * 16
    q, k = rows_out(s)
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


def test_streams_devices_and_graphs():
    """On a stream of its own, in a graph replayed over new rows, and with outputs that
    the call allocates there."""
    import paged_kv_cache_write_gb300 as pkv
    s = Step(50, 8, 2, 64, 64, "bf16", seed=9)
    ref = rows_out(s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = pkv.qk_norm_rope(s.q, s.k, *s.args, **s.kw_args, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    out = [torch.empty_like(t) for t in ref]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.qk_norm_rope(s.q, s.k, *s.args, **s.kw_args, q_out=out[0], k_out=out[1])
    s.qkv.copy_(-s.qkv)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(-a, b) for a, b in zip(ref, out))


def test_no_tokens():
    import paged_kv_cache_write_gb300 as pkv
    s = Step(0, 4, 2, 64, 64, "bf16")
    q, k = pkv.qk_norm_rope(s.q, s.k, *s.args, **s.kw_args)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
