"""The 4-bit cache in numpy float64: quantising write, the float64 value of every
element, and the norm and rotation that come before the cache.

An element stands for e2m1 x s x g: its four-bit code, the e4m3 scale of the 16
elements of its row that it is one of, and its KV head's scale.
"""
from __future__ import annotations

import numpy as np

from .paged_fp8 import E4M3, e4m3_encode  # noqa: F401

GROUP = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_encode(x: np.ndarray) -> np.ndarray:
    """Codes of the nearest e2m1 values, ties to the even code, 6 at most; the sign
    of zero is kept."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), E2M1[-1])
    d = np.abs(a[..., None] - E2M1)
    best = d.min(axis=-1, keepdims=True)
    even = np.where((d == best) & (np.arange(8) % 2 == 0), 1, 0)
    pick = np.where(even.any(axis=-1), even.argmax(axis=-1), (d == best).argmax(axis=-1))
    return (pick | (np.signbit(x).astype(np.int64) << 3)).astype(np.uint8)


def quantise(x, scale):
    """x float64 [..., n_kv, head_dim], scale [n_kv]: (packed codes [..., head_dim / 2],
    e4m3 bytes [..., head_dim / 16])."""
    x = np.asarray(x, dtype=np.float64)
    g = np.asarray(scale, dtype=np.float64)[:, None, None]
    y = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP) / g
    a = np.abs(y).max(axis=-1)  # NaN if one is
    s8 = e4m3_encode(a / 6.0)
    s = E4M3[s8][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, y / s, np.copysign(0.0, y))
    q = np.where(np.isnan(q), 0.0, q)  # (of a NaN group: any code)
    c = e2m1_encode(q).reshape(x.shape)
    return c[..., 0::2] | (c[..., 1::2] << 4), s8


def kv_write_fp4(x, slots, pool, groups, scale):
    """One of K / V.  x float64 [T, n_kv, hd], slots [T] (negative: skipped), pool uint8
    [nb, n_kv, bs, hd / 2], groups uint8 [nb, n_kv, bs, hd / 16]; returns both after the
    write."""
    pool, groups = pool.copy(), groups.copy()
    bs = pool.shape[2]
    if len(slots):
        codes, s8 = quantise(x, scale)
        for t, slot in enumerate(slots):
            if slot >= 0:
                pool[slot // bs, :, slot % bs] = codes[t]
                groups[slot // bs, :, slot % bs] = s8[t]
    return pool, groups


def values(pool, groups, scale) -> np.ndarray:
    """float64 [nb, bs, n_kv, hd]: the value of every element of a 4-bit pool."""
    signed = np.concatenate([E2M1, -E2M1])
    x = np.stack([signed[pool & 15], signed[pool >> 4]], axis=-1).reshape(*pool.shape[:-1], 2 * pool.shape[-1])
    x = x * np.repeat(E4M3[groups], GROUP, axis=-1)
    return (x * np.asarray(scale, dtype=np.float64)[:, None, None]).transpose(0, 2, 1, 3)


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """x float64 [T, heads, hd]: each head's row over its root mean square times the
    weight (None: as it is), then turned by its position's angles."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * weight
    row = np.asarray(cos_sin, dtype=np.float64)[positions][:, None, :]
    half = row.shape[-1] // 2
    c, s = row[..., :half], row[..., half:]
    y = x.copy()
    lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
              else (slice(0, half), slice(half, 2 * half)))
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y
