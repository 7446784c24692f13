"""The 8-bit cache in numpy float64: quantising write, read-back, and the
float64 value of every element, from which oracle.paged's attention follows.

An element stands for its e4m3 value times the power-of-two scale of its
(block, KV head).  e4m3 here is the 8-bit format with 4 exponent bits (bias 7),
3 mantissa bits, no infinities and NaN at 0x7f / 0xff.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
SCALE_MIN, SCALE_MAX = 2.0 ** -60, 2.0 ** 60


def _decode_byte(b: int) -> float:
    sign = -1.0 if b & 0x80 else 1.0
    e, m = (b >> 3) & 15, b & 7
    if e == 15 and m == 7:
        return float("nan")
    if e == 0:
        return sign * m * 2.0 ** -9
    return sign * (8 + m) * 2.0 ** (e - 10)


E4M3 = np.array([_decode_byte(b) for b in range(256)])
_POS = E4M3[:127]  # the finite values from 0 up, one per byte


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Bytes of the nearest e4m3 values, ties to the even byte; past 448 the
    largest value, NaN 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.searchsorted(_POS, a, side="left")          # first value >= a
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - _POS[lo], _POS[hi] - a
    pick = np.where(dhi < dlo, hi, np.where(dlo < dhi, lo, np.where(hi % 2 == 0, hi, lo)))
    out = (pick | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), out)


def scale_for(a: float) -> float:
    """Smallest power of two s in range with a <= 448 s."""
    s = SCALE_MIN
    while a > E4M3_MAX * s and s < SCALE_MAX:
        s *= 2.0
    return s


def kv_write_fp8(x, pool, scales, block_tables, seq_lens, new_lens):
    """One of K / V.  x float64 [T, n_kv, hd], pool uint8 [nb, bs, n_kv, hd],
    scales float64 [nb, n_kv]; returns the pool and scales after the write."""
    pool, scales = pool.copy(), scales.astype(np.float64).copy()
    bs, n_kv = pool.shape[1], pool.shape[2]
    t = 0
    for b, (L, n) in enumerate(zip(seq_lens, new_lens)):
        L, n = int(L), int(n)
        p = L - n
        while p < L:
            j, off = p // bs, p % bs
            m = min(bs - off, L - p)
            blk = int(block_tables[b, j])
            for h in range(n_kv):
                rows = x[t:t + m, h]
                mag = np.abs(rows[~np.isnan(rows)])
                s = scale_for(float(mag.max()) if mag.size else 0.0)
                if off > 0:
                    old = scales[blk, h]
                    s = max(s, old)
                    if s != old:
                        pool[blk, :off, h] = e4m3_encode(E4M3[pool[blk, :off, h]] * (old / s))
                with np.errstate(invalid="ignore"):
                    pool[blk, off:off + m, h] = e4m3_encode(rows / s)
                scales[blk, h] = s
            p += m
            t += m
    return pool, scales


def values(pool, scales) -> np.ndarray:
    """float64 value of every element of an 8-bit pool."""
    return E4M3[pool] * np.asarray(scales, dtype=np.float64)[:, None, :, None]
