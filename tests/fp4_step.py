"""Shared by the 4-bit cache's GPU tests: batches drawn from a seed, the float64
oracle on them, and the attention tolerance."""
import numpy as np
import torch

from gpu_step import check_canaries, guarded_copy, guarded_empty
from oracle import paged_fp4
from workloads import _blocks_held

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# half a step of a rounding, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def ints(x, dtype=np.int32):
    return guarded_copy(torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=dtype))))


class Batch:
    """Sequences with their tables over a 4-bit cache on the GPU, and the same cache in
    numpy.  What no token has written holds `garbage`: NaN scales under codes of 6."""

    def __init__(self, lens, *, n_kv, head_dim, dtype="bf16", block_size=16, spare=3, seed=0,
                 garbage=(0x77, 0x7F), num_blocks=None, scale=None):
        import paged_kv_cache_write_gb300 as pkv
        self.pkv = pkv
        self.lens = np.asarray(lens, dtype=np.int32)
        self.n_kv, self.hd, self.bs = n_kv, head_dim, block_size
        self.dtype = TYPES[dtype]
        self.g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        held = [_blocks_held(n, block_size) for n in self.lens]
        self.nb = num_blocks or sum(held) + spare
        ids = rng.permutation(self.nb)[: sum(held)]
        self.table = np.full((len(held), max(1, max(held, default=0))), self.nb - 1, dtype=np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = ids[at: at + n]
            at += n
        row = (self.nb, n_kv, block_size)
        self.kp, self.vp = (np.full((*row, head_dim // 2), garbage[0], dtype=np.uint8) for _ in range(2))
        self.kg, self.vg = (np.full((*row, head_dim // 16), garbage[1], dtype=np.uint8) for _ in range(2))
        if scale is None:  # heads of different powers of two
            self.ks, self.vs = (2.0 ** rng.integers(-7, 0, n_kv) for _ in range(2))
        else:
            self.ks, self.vs = (np.full(n_kv, scale, dtype=np.float64) for _ in range(2))
        self.d_kp, self.d_vp = (guarded_copy(torch.from_numpy(x)) for x in (self.kp, self.vp))
        self.d_kg, self.d_vg = (guarded_copy(torch.from_numpy(x).view(torch.float8_e4m3fn))
                                for x in (self.kg, self.vg))
        self.d_ks, self.d_vs = (guarded_copy(torch.from_numpy(x).float()) for x in (self.ks, self.vs))
        self.bt = guarded_copy(torch.from_numpy(self.table))
        self.err = guarded_empty((1,), torch.int32)
        self.err.zero_()

    @property
    def cache(self):
        return self.d_kp, self.d_vp, self.d_kg, self.d_vg, self.d_ks, self.d_vs

    def draw(self, tokens, mag=1.0, heads=None):
        """[tokens, heads, head_dim] with heads and channels of unequal size."""
        heads = heads or self.n_kv
        x = torch.randn(tokens, heads, self.hd, generator=self.g)
        x = x * torch.exp2(torch.randint(-3, 4, (heads, 1), generator=self.g).float())
        return (x * mag).to(self.dtype)

    def slots(self, lens, new):
        """Slot of each of the last new[b] of lens[b] tokens."""
        out = [self.table[b, p // self.bs] * self.bs + p % self.bs
               for b, (n, c) in enumerate(zip(lens, new)) for p in range(n - c, n)]
        return np.asarray(out, dtype=np.int64)

    def write(self, slots, k, v, err=None):
        """Both caches take the step; the GPU's is not compared here."""
        self.pkv.kv_write_fp4(guarded_copy(k), guarded_copy(v), ints(slots, np.int64), *self.cache,
                              err=self.err if err is None else err)
        check_canaries()
        self.take(slots, f64(k), f64(v))

    def take(self, slots, k, v):
        self.kp, self.kg = paged_fp4.kv_write_fp4(k, slots, self.kp, self.kg, self.ks)
        self.vp, self.vg = paged_fp4.kv_write_fp4(v, slots, self.vp, self.vg, self.vs)

    def fill(self, mag=1.0):
        """Every sequence's tokens written in one call."""
        t = int(self.lens.sum())
        if t:
            self.write(self.slots(self.lens, self.lens), self.draw(t, mag), self.draw(t, mag))

    def assert_same_cache(self):
        torch.cuda.synchronize()
        for p, g, rp, rg in ((self.d_kp, self.d_kg, self.kp, self.kg), (self.d_vp, self.d_vg, self.vp, self.vg)):
            p, g = p.cpu().numpy(), g.view(torch.uint8).cpu().numpy()
            nan = (rg & 0x7F) == 0x7F  # (a NaN has two bytes, and any codes)
            assert np.array_equal((g & 0x7F) == 0x7F, nan)
            assert np.array_equal(g[~nan], rg[~nan])
            fine = ~np.repeat(nan, 8, axis=-1)
            assert np.array_equal(p[fine], rp[fine])

    def rows(self, b, n):
        """float64 K, V [n, n_kv, hd] of sequence b's first n tokens."""
        blocks = self.table[b, : _blocks_held(n, self.bs)]
        return tuple(paged_fp4.values(p[blocks], g[blocks], s).reshape(-1, self.n_kv, self.hd)[:n]
                     for p, g, s in ((self.kp, self.kg, self.ks), (self.vp, self.vg, self.vs)))

    def reference(self, q, b, last, held=4):
        """(output, tolerance) [H, hd] in float64 of one query over keys 0..last.

        Tolerance, to first order.  The output is g sum(w v) / sum(w).  Scores are
        fp32 sums of at most 2 head_dim + 8 products (queries in two terms; keys are
        exact), so a score in log2 units is off by at most (2 head_dim + 8) 2^-24 S
        with S the sum of the products' magnitudes, and a weight relatively by ln 2
        times that, plus 2^-20 for the reference's subtraction at magnitudes up to 2^3
        and exp2, plus its own rounding: 2^-11 (f16) for bf16, 2^-21 (two f16 terms)
        for fp32.  Numerator and denominator each have the weights' error; the output
        is then rounded (half a step).

        f16 has an absolute floor besides: a weight below 2^-14 is rounded by up to
        2^-25.  Weights are held with their largest at 2^held or more (parts and
        earlier blocks, whose largest is smaller, count for less), so the numerator is
        off by at most 2^-(25 + held) max(p) sum |v| with p normalised.  A query row is
        held with its largest element at 2^14 or more, and an element below 2^-14
        there is rounded by up to 2^-25: a score is off by at most 2^-39 max |q| sum |k|.
        """
        K, V = self.rows(b, last + 1)
        H = q.shape[0]
        rep = H // self.n_kv
        scale = 1.0 / np.sqrt(self.hd)
        out, tol = np.zeros((H, self.hd)), np.zeros((H, self.hd))
        own = {torch.bfloat16: 2.0 ** -11, torch.float32: 2.0 ** -21}[self.dtype]
        for h in range(H):
            if last < 0:
                continue
            k, v = K[:, h // rep], V[:, h // rep]
            s = scale * (k @ q[h])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[h] = p @ v
            S = scale * np.log2(np.e) * (np.abs(k) @ np.abs(q[h])).max()
            floor = scale * np.log2(np.e) * np.abs(q[h]).max() * np.abs(k).sum(axis=1).max()
            rel = (np.log(2) * ((2 * self.hd + 8) * 2.0 ** -24 * S + 2.0 ** -39 * floor)
                   + 2.0 ** -20 * max(1.0, S / 8) + own)
            tol[h] = (HALF[self.dtype] * np.abs(out[h]) + 2 * rel * (p @ np.abs(v))
                      + 2.0 ** -(25 + held) * p.max() * np.abs(v).sum(axis=0) + 1e-30)
        return out, tol

    def check(self, got, q, which, last, held=4):
        """got, q [rows, H, hd]; row i is sequence which[i]'s, over keys 0..last[i].
        held: log2 of what a row's largest weight is held at or above."""
        got, q = f64(got), f64(q)
        worst = 0.0
        for i, (b, n) in enumerate(zip(which, last)):
            ref, tol = self.reference(q[i], b, n, held)
            assert np.all(np.isfinite(got[i])), (i, b, n)
            worst = max(worst, float(np.max(np.abs(got[i] - ref) / tol)) if n >= 0
                        else float(np.abs(got[i]).max()))
        assert worst <= 1.0, worst

    def decode(self, q, lens=None, max_ctas=0, **kw):
        lens = self.lens if lens is None else np.asarray(lens, dtype=np.int32)
        out = self.pkv.paged_attention_decode_fp4(
            guarded_copy(q), *self.cache, self.bt, ints(lens), 1.0 / np.sqrt(self.hd),
            int(max(0, lens.max(initial=0))), out=guarded_empty(q.shape, q.dtype),
            workspace=guarded_empty((self.pkv.decode_fp4_workspace_bytes(
                q.shape[0], q.shape[1], self.hd, int(lens.max(initial=0)), max_ctas),), torch.uint8),
            max_ctas=max_ctas, err=self.err, **kw)
        check_canaries()
        return out

    def prefill(self, q, lens, new, **kw):
        lens, new = np.asarray(lens, dtype=np.int32), np.asarray(new, dtype=np.int32)
        cu = np.concatenate([[0], np.cumsum(new)])
        out = self.pkv.paged_attention_prefill_fp4(
            guarded_copy(q), ints(cu), *self.cache, self.bt, ints(lens), 1.0 / np.sqrt(self.hd),
            int(new.max()), int(lens.max()), out=guarded_empty(q.shape, q.dtype), err=self.err, **kw)
        check_canaries()
        return out

    def queries(self, rows, heads, mag=1.5):
        return (mag * torch.randn(rows, heads, self.hd, generator=self.g)).to(self.dtype)

    def no_error(self):
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
