"""The 4-bit cache and the norm and rotation on the CPU: their oracle against closed
forms, and the entry points' refusals (host checks that run before any launch and
never touch a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged_fp4

FAKE = 0x10000  # a 16-byte-aligned non-null address; never dereferenced
F32, BF16 = 0, 1
OK, NULL, SHAPE, DTYPE, ALIGN, RANGE, WORKSPACE, UNSUPPORTED = range(8)


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_write_gb300 import build
    build.build()
    import paged_kv_cache_write_gb300 as m
    return m


# ------------------------------------------------------------------ oracle

def test_codes_are_nearest_even():
    v = paged_fp4.E2M1
    assert list(paged_fp4.e2m1_encode(v)) == list(range(8))
    assert list(paged_fp4.e2m1_encode(-v)) == list(range(8, 16))
    mid = (v[1:] + v[:-1]) / 2
    assert list(paged_fp4.e2m1_encode(mid)) == [0, 2, 2, 4, 4, 6, 6]
    assert list(paged_fp4.e2m1_encode(np.nextafter(mid, 9))) == list(range(1, 8))
    assert list(paged_fp4.e2m1_encode(np.nextafter(mid, 0))) == list(range(7))
    assert list(paged_fp4.e2m1_encode(np.array([6.5, 1e30, np.inf, -np.inf]))) == [7, 7, 7, 15]


def test_quantising_is_off_by_half_a_code_step():
    """|x - value| <= scale x half the widest gap between codes that it lies between,
    plus what the scale's own rounding cuts off at 6."""
    rng = np.random.default_rng(0)
    x = rng.normal(size=(50, 3, 64))
    g = np.array([0.25, 1.0, 0.125])
    codes, s8 = paged_fp4.quantise(x, g)
    back = paged_fp4.values(codes[:, :, None], s8[:, :, None], g)[:, 0]
    s = np.repeat(paged_fp4.E4M3[s8], 16, axis=-1) * g[:, None]
    q = np.abs(x) / s
    gap = np.where(q < 2, 0.25, np.where(q < 4, 0.5, 1.0))
    assert np.all(np.abs(x - back) <= s * gap * (1 + 1e-12))
    assert q.max() <= 6 * (1 + 2.0 ** -4)  # e4m3 rounds by 2^-4 at most
    codes, s8 = paged_fp4.quantise(back, g)  # quantised values whose scale is a code stay
    again = paged_fp4.values(codes[:, :, None], s8[:, :, None], g)[:, 0]
    full = np.abs(back).reshape(50, 3, 4, 16).max(-1) == 6 * paged_fp4.E4M3[s8] * g[:, None]
    assert np.array_equal(back.reshape(50, 3, 4, 16)[full], again.reshape(50, 3, 4, 16)[full])


def test_layout_of_pools():
    x = np.arange(-8, 8, dtype=np.float64)[None, None, :].repeat(2, axis=1)
    pool, groups = np.zeros((2, 2, 4, 8), np.uint8), np.zeros((2, 2, 4, 1), np.uint8)
    pool, groups = paged_fp4.kv_write_fp4(x, [6], pool, groups, np.array([1.0, 2.0]))
    assert not pool[0].any() and not pool[1, :, [0, 1, 3]].any()
    v = paged_fp4.values(pool, groups, np.array([1.0, 2.0]))
    assert v.shape == (2, 4, 2, 16) and v[1, 2, 0, 0] < 0 < v[1, 2, 0, 15]
    # 8 / 6 lies between 1.25 and 1.375 (e4m3): 1.375; 7 / 1.375 = 5.09 goes to 6
    assert groups[1, 0, 2, 0] == 0x3B and v[1, 2, 0, 15] == 6 * 1.375
    assert pool[1, 0, 2, 7] >> 4 == 7  # element 15 in the high half of the last byte


def test_norm_and_rotation_against_closed_forms():
    x = np.random.default_rng(1).normal(size=(3, 2, 32))
    still = np.concatenate([np.ones((4, 8)), np.zeros((4, 8))], axis=1)
    assert np.array_equal(paged_fp4.norm_rope(x, None, 0.0, still, [0, 1, 2], False), x)
    y = paged_fp4.norm_rope(x, np.ones(32), 0.0, still, [0, 0, 0], True)
    assert np.allclose((y * y).mean(-1), 1.0)
    quarter = np.concatenate([np.zeros((1, 8)), np.ones((1, 8))], axis=1)
    y = paged_fp4.norm_rope(x, None, 0.0, quarter, [0, 0, 0], False)
    assert np.array_equal(y[..., :8], -x[..., 8:16]) and np.array_equal(y[..., 8:16], x[..., :8])
    assert np.array_equal(y[..., 16:], x[..., 16:])
    y = paged_fp4.norm_rope(x, None, 0.0, quarter, [0, 0, 0], True)
    assert np.array_equal(y[..., 0:16:2], -x[..., 1:16:2]) and np.array_equal(y[..., 1:16:2], x[..., 0:16:2])
    # a product of a turned query and a turned key depends on the difference of positions
    a = np.arange(20)[:, None] * 0.7 ** np.arange(8)
    cs = np.concatenate([np.cos(a), np.sin(a)], axis=1)
    dot = [(paged_fp4.norm_rope(x[:1], None, 0, cs, [p], False)
            * paged_fp4.norm_rope(x[1:2], None, 0, cs, [p + 5], False)).sum() for p in (0, 3, 14)]
    assert np.allclose(dot, dot[0])


# ---------------------------------------------------------------- refusals

class Calls:
    """One good call of each entry; a keyword changes one of its arguments."""

    def __init__(self, pkv):
        self.pkv, self.lib = pkv, pkv.lib

    def rope(self, **kw):
        d = dict(q_weight=FAKE, k_weight=FAKE, eps=1e-6, rot_dim=64, interleaved=0, num_positions=9,
                 cos_sin=FAKE, positions=FAKE)
        d.update({k: kw.pop(k) for k in list(kw) if k in d})
        return self.pkv.NormRopeDesc(*d.values())

    def desc(self, kw, dtype):
        d = dict(num_blocks=8, block_size=16, n_kv=2, head_dim=64, dtype=dtype)
        d.update({k: kw.pop(k) for k in list(kw) if k in d})
        return self.pkv.PoolDesc(*d.values())

    @staticmethod
    def fill(d, kw):
        assert set(kw) <= set(d), kw
        d.update(kw)
        return list(d.values())

    def rows(self, **kw):
        r = {k: kw.pop(k) for k in list(kw) if k in ("q_weight", "k_weight", "eps", "rot_dim", "interleaved",
                                                     "num_positions", "cos_sin", "positions")}
        rope = None if kw.pop("no_rope", False) else ctypes.byref(self.rope(**r))
        return self.lib.pkv_qk_norm_rope(*self.fill(dict(
            q=FAKE, qs=256, k=FAKE, ks=128, dtype=BF16, T=0, H=4, n_kv=2, hd=64, rope=rope, qo=FAKE, qos=256,
            ko=FAKE, kos=128), kw), None, None)

    def write(self, **kw):
        r = {k: kw.pop(k) for k in list(kw) if k in ("eps", "rot_dim", "interleaved", "num_positions",
                                                     "cos_sin", "positions")}
        d = None if kw.pop("no_pool", False) else ctypes.byref(self.desc(kw, kw.pop("pool_dtype", BF16)))
        return self.lib.pkv_qk_norm_rope_write(*self.fill(dict(
            q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, T=0, H=4, rope=ctypes.byref(self.rope(**r)), qo=FAKE,
            qos=256, slots=FAKE, kp=FAKE, vp=FAKE, pool=d), kw), None, None)

    def write_both(self, **kw):
        d = self.desc(kw, kw.pop("pool_dtype", 3))
        return self.lib.pkv_qk_norm_rope_write_fp4(*self.fill(dict(
            q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, type=BF16, T=0, H=4, rope=ctypes.byref(self.rope()),
            qo=FAKE, qos=256, slots=FAKE, kp=FAKE, vp=FAKE, kg=FAKE, vg=FAKE, k1=FAKE, v1=FAKE,
            pool=ctypes.byref(d)), kw), None, None)

    def write_fp4(self, **kw):
        d = None if kw.pop("no_pool", False) else ctypes.byref(self.desc(kw, kw.pop("pool_dtype", 3)))
        return self.lib.pkv_kv_write_fp4(*self.fill(dict(
            k=FAKE, ks=128, v=FAKE, vs=128, type=BF16, slots=FAKE, T=0, kp=FAKE, vp=FAKE, kg=FAKE, vg=FAKE,
            k1=FAKE, v1=FAKE, pool=d), kw), None, None)

    def gather(self, **kw):
        d = None if kw.pop("no_pool", False) else ctypes.byref(self.desc(kw, kw.pop("pool_dtype", 3)))
        return self.lib.pkv_kv_gather_fp4(*self.fill(dict(
            kp=FAKE, vp=FAKE, kg=FAKE, vg=FAKE, k1=FAKE, v1=FAKE, pool=d, bt=FAKE, W=4, lens=FAKE, cu=FAKE, B=2,
            total=0, type=BF16, ko=FAKE, vo=FAKE), kw), None, None)


BIG = 1 << 62


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(no_rope=True), NULL), (dict(dtype=2), DTYPE), (dict(T=-1), SHAPE),
    (dict(H=0), SHAPE), (dict(n_kv=0), SHAPE), (dict(hd=0), SHAPE), (dict(hd=72), UNSUPPORTED),
    (dict(hd=272, rot_dim=16), UNSUPPORTED), (dict(rot_dim=0), SHAPE), (dict(rot_dim=80), SHAPE),
    (dict(rot_dim=24), UNSUPPORTED), (dict(num_positions=0), SHAPE), (dict(interleaved=2), RANGE),
    (dict(eps=-1.0), RANGE), (dict(eps=float("nan")), RANGE), (dict(eps=float("inf")), RANGE),
    (dict(eps=-1.0, q_weight=None, k_weight=None), OK),
    (dict(T=3, cos_sin=None), NULL), (dict(T=3, positions=None), NULL), (dict(T=3, cos_sin=FAKE + 8), ALIGN),
    (dict(T=3, positions=FAKE + 2), ALIGN), (dict(T=3, q_weight=FAKE + 2), ALIGN),
    (dict(T=3, q=None), NULL), (dict(T=3, k=None), NULL), (dict(T=3, qo=None), NULL), (dict(T=3, ko=None), NULL),
    (dict(T=3, q=FAKE + 8), ALIGN), (dict(T=3, qs=255), SHAPE), (dict(T=3, qs=260), ALIGN),
    (dict(T=3, ks=-128), SHAPE), (dict(T=3, kos=127), SHAPE), (dict(T=3, ko=FAKE + 4), ALIGN),
    (dict(T=3, qos=BIG), RANGE), (dict(T=(1 << 31) - 1, H=1 << 20, qs=1 << 27, qos=1 << 27), RANGE),
    (dict(T=3, H=1 << 30, qs=1 << 36, qos=1 << 36), RANGE)])
def test_norm_rope_refusals(pkv, kw, status):
    assert Calls(pkv).rows(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(no_pool=True), NULL), (dict(pool_dtype=2), DTYPE), (dict(pool_dtype=3), DTYPE),
    (dict(num_blocks=0), SHAPE), (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(head_dim=72), UNSUPPORTED),
    (dict(T=3, v=None), NULL), (dict(T=3, slots=None), NULL), (dict(T=3, kp=None), NULL),
    (dict(T=3, vp=FAKE + 8), ALIGN), (dict(T=3, slots=FAKE + 4), ALIGN), (dict(T=3, vs=64), SHAPE),
    (dict(T=3, vs=132), ALIGN), (dict(rot_dim=128), SHAPE)])
def test_norm_rope_write_refusals(pkv, kw, status):
    assert Calls(pkv).write(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(pool_dtype=1), DTYPE), (dict(type=3), DTYPE), (dict(T=-1), SHAPE), (dict(H=0), SHAPE),
    (dict(T=3, kg=None), NULL), (dict(T=3, v1=None), NULL), (dict(T=3, vg=FAKE + 4), ALIGN),
    (dict(T=3, k1=FAKE + 2), ALIGN), (dict(T=3, vp=None), NULL)])
def test_norm_rope_write_fp4_refusals(pkv, kw, status):
    assert Calls(pkv).write_both(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(no_pool=True), NULL), (dict(pool_dtype=1), DTYPE), (dict(type=2), DTYPE),
    (dict(T=-1), SHAPE), (dict(n_kv=0), SHAPE), (dict(head_dim=24), UNSUPPORTED),
    (dict(head_dim=272), UNSUPPORTED), (dict(n_kv=65536), RANGE), (dict(num_blocks=1 << 30), RANGE),
    (dict(num_blocks=1 << 26, n_kv=32), RANGE),
    (dict(T=3, k=None), NULL), (dict(T=3, v=None), NULL), (dict(T=3, slots=None), NULL),
    (dict(T=3, kp=None), NULL), (dict(T=3, vp=None), NULL), (dict(T=3, kg=None), NULL),
    (dict(T=3, vg=None), NULL), (dict(T=3, k1=None), NULL), (dict(T=3, v1=None), NULL),
    (dict(T=3, k=FAKE + 8), ALIGN), (dict(T=3, kp=FAKE + 8), ALIGN), (dict(T=3, kg=FAKE + 8), ALIGN),
    (dict(T=3, ks=100), SHAPE), (dict(T=3, ks=132), ALIGN),
    (dict(T=(1 << 31) - 1, n_kv=65535, ks=1 << 25, vs=1 << 25), RANGE)])
def test_write_refusals(pkv, kw, status):
    assert Calls(pkv).write_fp4(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(no_pool=True), NULL), (dict(pool_dtype=0), DTYPE), (dict(type=2), DTYPE),
    (dict(B=-1), SHAPE), (dict(total=-1), SHAPE), (dict(W=-1), SHAPE), (dict(total=5, B=0), SHAPE),
    (dict(total=5, W=0), SHAPE), (dict(total=5, kp=None), NULL), (dict(total=5, vg=None), NULL),
    (dict(total=5, k1=None), NULL), (dict(total=5, bt=None), NULL), (dict(total=5, lens=None), NULL),
    (dict(total=5, cu=None), NULL), (dict(total=5, vo=None), NULL), (dict(total=5, ko=FAKE + 8), ALIGN),
    (dict(total=5, kg=FAKE + 8), ALIGN), (dict(total=5, v1=FAKE + 1), ALIGN)])
def test_gather_refusals(pkv, kw, status):
    assert Calls(pkv).gather(**kw) == status


def test_other_entries_refuse_4_bit_pools(pkv):
    d = ctypes.byref(pkv.PoolDesc(8, 16, 2, 64, 3))
    assert pkv.lib.pkv_kv_write(FAKE, FAKE, FAKE, 0, FAKE, FAKE, d, None, None) == DTYPE
    assert pkv.lib.pkv_kv_gather_fp8(FAKE, FAKE, FAKE, FAKE, d, FAKE, 4, FAKE, FAKE, 2, 0, 1, FAKE, FAKE, None,
                                     None) == DTYPE


def test_binding_refuses_mismatched_tensors(pkv):
    """On the CPU: every call needs tensors on a GPU, and says so."""
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkv.qk_norm_rope(x, x, torch.zeros(4, 64), torch.zeros(2, dtype=torch.int32))
    pool, groups = torch.zeros(2, 4, 16, 32, dtype=torch.uint8), torch.zeros(2, 4, 16, 4).to(torch.float8_e4m3fn)
    scale = torch.ones(4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkv.kv_write_fp4(x, x, torch.zeros(2, dtype=torch.int64), pool, pool, groups, groups, scale, scale)
    with pytest.raises(ValueError, match="one per 16 elements"):
        pkv.kv_write_fp4(x, x, torch.zeros(2, dtype=torch.int64), pool, pool, groups[:1], groups, scale, scale)
    with pytest.raises(ValueError, match="one per KV head"):
        pkv.kv_write_fp4(x, x, torch.zeros(2, dtype=torch.int64), pool, pool, groups, groups, scale[:1], scale)
    with pytest.raises(ValueError, match="same shape"):
        pkv.kv_write_fp4(x, x, torch.zeros(2, dtype=torch.int64), pool, pool[:1], groups, groups, scale, scale)


class Attention(Calls):
    def decode(self, **kw):
        d = None if kw.pop("no_pool", False) else ctypes.byref(self.desc(kw, kw.pop("pool_dtype", 3)))
        return self.lib.pkv_paged_attention_decode_fp4(*self.fill(dict(
            q=FAKE, type=BF16, B=2, H=8, kp=FAKE, vp=FAKE, kg=FAKE, vg=FAKE, k1=FAKE, v1=FAKE, pool=d, bt=FAKE,
            W=4, lens=FAKE, most=64, scale=0.1, ctas=0, out=FAKE, ws=FAKE, ws_bytes=1, err=None, stream=None), kw))

    def prefill(self, **kw):
        d = None if kw.pop("no_pool", False) else ctypes.byref(self.desc(kw, kw.pop("pool_dtype", 3)))
        return self.lib.pkv_paged_attention_prefill_fp4(*self.fill(dict(
            q=FAKE, type=BF16, cu=FAKE, B=2, total=0, most_q=8, H=8, kp=FAKE, vp=FAKE, kg=FAKE, vg=FAKE, k1=FAKE,
            v1=FAKE, pool=d, bt=FAKE, W=4, lens=FAKE, most=64, scale=0.1, out=FAKE, err=None, stream=None), kw))


COMMON = [
    (dict(no_pool=True), NULL), (dict(pool_dtype=1), DTYPE), (dict(type=2), DTYPE), (dict(B=-1), SHAPE),
    (dict(H=0), SHAPE), (dict(H=7), SHAPE), (dict(W=-1), SHAPE), (dict(most=-1), SHAPE), (dict(most=65), SHAPE),
    (dict(scale=0.0), RANGE), (dict(scale=float("inf")), RANGE), (dict(scale=float("nan")), RANGE),
    (dict(q=None), NULL), (dict(kp=None), NULL), (dict(vp=None), NULL), (dict(kg=None), NULL),
    (dict(vg=None), NULL), (dict(k1=None), NULL), (dict(v1=None), NULL), (dict(bt=None), NULL),
    (dict(lens=None), NULL), (dict(out=None), NULL), (dict(q=FAKE + 8), ALIGN), (dict(kp=FAKE + 8), ALIGN),
    (dict(kg=FAKE + 8), ALIGN), (dict(k1=FAKE + 2), ALIGN), (dict(out=FAKE + 4), ALIGN),
    (dict(head_dim=48), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(block_size=32), UNSUPPORTED),
    (dict(H=34), UNSUPPORTED), (dict(W=1 << 27), RANGE), (dict(n_kv=65536, H=65536), RANGE)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(ctas=-1), RANGE), (dict(B=1 << 20, n_kv=64, H=64, most=16 * 64, W=64), RANGE),
    (dict(B=1 << 30, n_kv=8), RANGE), (dict(ws=None), WORKSPACE), (dict(), WORKSPACE),
    (dict(ws=FAKE + 8, ws_bytes=1 << 50), ALIGN), (dict(B=0, q=None, ws=None), OK)])
def test_decode_refusals(pkv, kw, status):
    assert Attention(pkv).decode(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(), OK), (dict(total=-1), SHAPE), (dict(most_q=-1), SHAPE), (dict(total=9, cu=None), NULL),
    (dict(total=9, most_q=0), SHAPE), (dict(total=7, most_q=8), SHAPE), (dict(total=99, most_q=65), SHAPE),
    (dict(B=0, q=None), OK)])
def test_prefill_refusals(pkv, kw, status):
    assert Attention(pkv).prefill(**kw) == status


def test_workspace_sizes(pkv):
    a = pkv.decode_fp4_workspace_bytes(4, 8, 64, 100)
    assert a > 0 and pkv.decode_fp4_workspace_bytes(8, 8, 128, 100) > a
    assert pkv.decode_fp4_workspace_bytes(-1, 0, 0, 0) > 0
