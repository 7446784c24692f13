"""The 8-bit cache on the CPU: its oracle against closed forms and the e4m3
format, and the entry points' refusals (host checks that run before any
launch and never touch a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged_fp8

FAKE = 0x10000  # a 16-byte-aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_write_gb300 import build
    build.build()
    import paged_kv_cache_write_gb300 as m
    return m


# ------------------------------------------------------------------ oracle

def test_byte_values_are_torchs():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
    ref = t.float().numpy().astype(np.float64)
    assert np.array_equal(paged_fp8.E4M3, ref, equal_nan=True)
    assert np.array_equal(np.signbit(paged_fp8.E4M3[:255]), np.signbit(ref[:255]))


def test_encode_is_nearest_even():
    # every value, every midpoint between neighbours, and just beside each
    v = paged_fp8.E4M3[:127]
    assert np.array_equal(paged_fp8.e4m3_encode(v), np.arange(127))
    mid = (v[1:] + v[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(paged_fp8.e4m3_encode(mid), even)
    assert np.array_equal(paged_fp8.e4m3_encode(np.nextafter(mid, 1e9)), np.arange(1, 127))
    assert np.array_equal(paged_fp8.e4m3_encode(-np.nextafter(mid, 0)), np.arange(126) | 0x80)
    x = np.random.default_rng(0).normal(size=4000) * 2.0 ** np.random.default_rng(1).integers(-12, 8, 4000)
    x = x[np.abs(x) <= 448]
    t = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    x32 = x.astype(np.float32).astype(np.float64)
    assert np.array_equal(paged_fp8.e4m3_encode(x32), t)
    got = paged_fp8.e4m3_encode(np.array([500.0, -1e9, np.inf, np.nan]))
    assert list(got) == [0x7E, 0xFE, 0x7E, 0x7F]


def test_scale_is_the_smallest_that_fits():
    for a in (448.0, 224.0, 1.0, 3.0, 1e-3, np.nextafter(448.0, 1e9), np.nextafter(448.0, 0)):
        s = paged_fp8.scale_for(a)
        assert a <= 448 * s and a > 448 * s / 2 and np.log2(s) == round(np.log2(s))
    assert paged_fp8.scale_for(0.0) == 2.0 ** -60
    assert paged_fp8.scale_for(np.inf) == 2.0 ** 60


def test_write_grows_a_blocks_scale_and_keeps_its_tokens():
    bs, n_kv, hd = 4, 1, 16
    pool = np.full((3, bs, n_kv, hd), 0x7F, dtype=np.uint8)
    scales = np.full((3, n_kv), 3.0)
    x = np.ones((3, n_kv, hd))
    x[2] = 1000.0
    table = np.array([[2, 1]])
    pool, scales = paged_fp8.kv_write_fp8(x[:2], pool, scales, table, [2], [2])
    assert scales[2, 0] == 2.0 ** -8
    pool2, scales2 = paged_fp8.kv_write_fp8(x[2:], pool, scales, table, [3], [1])
    assert scales2[2, 0] == 4.0
    v = paged_fp8.values(pool2, scales2)
    assert np.all(v[2, :2] == 1.0) and np.all(v[2, 2] == 1024.0)  # 250 is a tie: 256
    assert np.all(pool2[2, 3] == 0x7F) and np.all(pool2[[0, 1]] == 0x7F)


def test_rounding_error_is_at_most_half_a_step():
    """|value - x| <= 2^-4 |x| for e4m3's normal range, half a subnormal step below."""
    x = np.random.default_rng(5).normal(size=(16, 2, 32))
    pool, sc = paged_fp8.kv_write_fp8(x, np.zeros((1, 16, 2, 32), np.uint8), np.zeros((1, 2)),
                                      np.array([[0]]), [16], [16])
    v = paged_fp8.values(pool, sc)[0]
    bound = np.maximum(np.abs(x) * 2.0 ** -4, sc[0][None, :, None] * 2.0 ** -10)
    assert np.all(np.abs(v - x) <= bound)


# --------------------------------------------------------------- refusals

def _desc(pkv, **kw):
    d = dict(num_blocks=8, block_size=16, n_kv=2, head_dim=64, dtype=2)
    d.update(kw)
    return pkv.PoolDesc(**d)


def _write(pkv, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=1, bt=FAKE, W=4, sl=FAKE, cu=FAKE, B=2, T=3, kp=FAKE, vp=FAKE,
             ks=FAKE, vs=FAKE, desc=_desc(pkv))
    a.update(kw)
    d = a["desc"]
    return pkv.lib.pkv_kv_write_fp8(a["k"], a["v"], a["dtype"], a["bt"], a["W"], a["sl"], a["cu"],
                                    a["B"], a["T"], a["kp"], a["vp"], a["ks"], a["vs"],
                                    None if d is None else ctypes.byref(d), None, None)


def _gather(pkv, **kw):
    a = dict(kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, W=4, sl=FAKE, cu=FAKE, B=2, T=3, dtype=1,
             ko=FAKE, vo=FAKE, desc=_desc(pkv))
    a.update(kw)
    d = a["desc"]
    return pkv.lib.pkv_kv_gather_fp8(a["kp"], a["vp"], a["ks"], a["vs"],
                                     None if d is None else ctypes.byref(d), a["bt"], a["W"],
                                     a["sl"], a["cu"], a["B"], a["T"], a["dtype"], a["ko"], a["vo"],
                                     None, None)


@pytest.mark.parametrize("call", [_write, _gather], ids=["write", "gather"])
def test_write_and_gather_refusals(pkv, call):
    out = ("k", "v") if call is _write else ("ko", "vo")
    assert call(pkv, desc=None) == 1
    for dtype in (0, 1, 7):  # a pool that is not 8 bits wide
        assert call(pkv, desc=_desc(pkv, dtype=dtype)) == 3
    for dtype in (2, 7, -1):
        assert call(pkv, dtype=dtype) == 3
    for bad in (dict(num_blocks=0), dict(block_size=0), dict(n_kv=-1), dict(head_dim=0)):
        assert call(pkv, desc=_desc(pkv, **bad)) == 2
    assert call(pkv, desc=_desc(pkv, head_dim=40)) == 7
    assert call(pkv, desc=_desc(pkv, num_blocks=1 << 30)) == 5
    for bad in (dict(T=-1), dict(B=-1), dict(W=-1), dict(B=0), dict(W=0)):
        assert call(pkv, **bad) == 2
    for name in ("kp", "vp", "ks", "vs", "bt", "sl", "cu", *out):
        assert call(pkv, **{name: None}) == 1, name
    for name in ("kp", "vp", *out):
        assert call(pkv, **{name: FAKE + 8}) == 4, name
    for name in ("ks", "vs"):
        assert call(pkv, **{name: FAKE + 2}) == 4, name
    assert call(pkv, T=0, **{out[0]: None}) == 0  # nothing to do


def _decode(pkv, **kw):
    a = dict(q=FAKE, dtype=1, B=2, H=8, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, W=4, sl=FAKE,
             msl=64, scale=0.125, ctas=0, out=FAKE, ws=FAKE, wsb=1 << 40, desc=_desc(pkv))
    a.update(kw)
    d = a["desc"]
    return pkv.lib.pkv_paged_attention_decode_fp8(
        a["q"], a["dtype"], a["B"], a["H"], a["kp"], a["vp"], a["ks"], a["vs"],
        None if d is None else ctypes.byref(d), a["bt"], a["W"], a["sl"], a["msl"], a["scale"],
        a["ctas"], a["out"], a["ws"], a["wsb"], None, None)


def _prefill(pkv, **kw):
    a = dict(q=FAKE, dtype=1, cu=FAKE, B=2, T=10, mq=8, H=8, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE,
             bt=FAKE, W=4, sl=FAKE, msl=64, scale=0.125, out=FAKE, desc=_desc(pkv))
    a.update(kw)
    d = a["desc"]
    return pkv.lib.pkv_paged_attention_prefill_fp8(
        a["q"], a["dtype"], a["cu"], a["B"], a["T"], a["mq"], a["H"], a["kp"], a["vp"], a["ks"],
        a["vs"], None if d is None else ctypes.byref(d), a["bt"], a["W"], a["sl"], a["msl"],
        a["scale"], a["out"], None, None)


@pytest.mark.parametrize("call", [_decode, _prefill], ids=["decode", "prefill"])
def test_attention_refusals(pkv, call):
    assert call(pkv, desc=None) == 1
    for dtype in (0, 1, 7):
        assert call(pkv, desc=_desc(pkv, dtype=dtype)) == 3
    for dtype in (2, 7):
        assert call(pkv, dtype=dtype) == 3
    for bad in (dict(B=-1), dict(H=0), dict(H=9), dict(W=-1), dict(msl=-1), dict(msl=65), dict(W=0)):
        assert call(pkv, **bad) == 2, bad
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(pkv, scale=scale) == 5
    for name in ("q", "kp", "vp", "ks", "vs", "bt", "sl", "out"):
        assert call(pkv, **{name: None}) == 1, name
    for name in ("q", "kp", "vp", "out"):
        assert call(pkv, **{name: FAKE + 8}) == 4, name
    for bad in (dict(head_dim=48), dict(block_size=32), dict(head_dim=256)):
        assert call(pkv, desc=_desc(pkv, **bad)) == 7, bad
    assert call(pkv, H=34) == 7  # 17 query heads to a KV head
    assert call(pkv, B=0) == 0


def test_decode_refusals(pkv):
    assert _decode(pkv, ctas=-1) == 5
    assert _decode(pkv, ws=None) == 6
    need = pkv.decode_fp8_workspace_bytes(2, 8, 64, 64)
    assert need > 0 and _decode(pkv, wsb=need - 1) == 6
    assert _decode(pkv, ws=FAKE + 4) == 4


def test_prefill_refusals(pkv):
    for bad in (dict(T=-1), dict(mq=-1), dict(mq=0), dict(mq=11), dict(mq=65, T=100)):
        assert _prefill(pkv, **bad) == 2, bad
    assert _prefill(pkv, cu=None) == 1
    assert _prefill(pkv, T=0, mq=0) == 0


def test_other_entries_refuse_8_bit_pools(pkv):
    """An 8-bit pool without its scales is refused, not misread."""
    by = ctypes.byref
    d = _desc(pkv)
    assert pkv.lib.pkv_kv_write(FAKE, FAKE, FAKE, 4, FAKE, FAKE, by(d), None, None) == 3
    assert pkv.lib.pkv_paged_attention_decode(FAKE, 2, 8, FAKE, FAKE, by(d), FAKE, 4, FAKE, 64, 0.1,
                                              0, FAKE, FAKE, 1 << 40, None, None) == 3


def test_binding_refuses_mismatched_tensors(pkv):
    """Shape, type and placement checks of the binding (no CUDA tensor is
    ever accepted here: the last check refuses host memory)."""
    kp = torch.zeros(4, 16, 2, 64, dtype=torch.float8_e4m3fn)
    sc = torch.ones(4, 2)
    bt = torch.zeros(2, 3, dtype=torch.int32)
    sl = torch.ones(2, dtype=torch.int32)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    w = pkv.kv_write_fp8
    with pytest.raises(ValueError, match="k_scales"):
        w(k, k, bt, sl, cu, kp, kp, torch.ones(4), torch.ones(4))
    with pytest.raises(ValueError, match="same shape"):
        w(k, k, bt, sl, cu, kp, kp[:2], sc, sc)
    with pytest.raises(ValueError, match="CUDA tensor"):
        w(k, k, bt, sl, cu, kp, kp, sc, sc)
    q = torch.zeros(2, 4, 32, dtype=torch.bfloat16)
    if not torch.cuda.is_available():
        return
    kp, sc, bt, sl, cu, k = (t.cuda() for t in (kp, sc, bt, sl, cu, k))
    with pytest.raises(TypeError):
        w(k.half(), k.half(), bt, sl, cu, kp, kp, sc, sc)
    with pytest.raises(TypeError):
        w(k, k, bt, sl, cu, kp.view(torch.uint8), kp, sc, sc)
    with pytest.raises(ValueError, match="matching the pool"):
        w(k[:, :1], k[:, :1], bt, sl, cu, kp, kp, sc, sc)
    with pytest.raises(ValueError, match="cu_new_lens"):
        w(k, k, bt, sl, cu[:2], kp, kp, sc, sc)
    with pytest.raises(ValueError, match="contiguous"):
        w(k.transpose(0, 1).contiguous().transpose(0, 1), k, bt, sl, cu, kp, kp, sc, sc)
    with pytest.raises(ValueError, match="is on cpu"):
        w(k, k, bt, sl.cpu(), cu, kp, kp, sc, sc)
    with pytest.raises(ValueError, match="head_dim"):
        pkv.paged_attention_decode_fp8(q.cuda(), kp, kp, sc, sc, bt, sl, 0.1, 1)


def test_refusals_of_extents_past_32_bits(pkv):
    """Extents that the kernels count in 32 bits, one past what they hold."""
    for call in (_write, _gather):
        assert call(pkv, desc=_desc(pkv, n_kv=(1 << 20) + 1)) == 5
        assert call(pkv, desc=_desc(pkv, num_blocks=1, block_size=1 << 25)) == 5
    for call in (_decode, _prefill):
        assert call(pkv, W=1 << 27) == 5
        assert call(pkv, desc=_desc(pkv, n_kv=(1 << 20) + 1), H=(1 << 20) + 1) == 5
