"""Block-scaled FP8 pools without a GPU: the 64-bit restatement that the GPU
tests compare with is pinned here, and the host checks refuse bad arguments
before any CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_attention_prepare_gb300 as pa
import scaled_ref as ref
from helpers import dense_causal_numpy

FAKE = ctypes.c_void_p(0x100000)   # never dereferenced: the checks return first
ODD = ctypes.c_void_p(0x100004)


def test_reference_codes_match_the_oracle():
    every = np.arange(256, dtype=np.uint8)
    a, b = ref.decode(every), oracle.e4m3_decode(every)
    np.testing.assert_array_equal(np.isnan(a), np.isnan(b))
    ok = ~np.isnan(a)
    np.testing.assert_array_equal(a[ok], b[ok])
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 12, 20000)).astype(np.float32)
    x = np.concatenate([x, ref._MID, -ref._MID, ref.POSITIVE, [0.0, 1e9, -1e9]]).astype(np.float32)
    np.testing.assert_array_equal(ref.encode(x), oracle.e4m3_encode(x))


@pytest.mark.parametrize("amax,e", [(0.0, -56), (448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0),
                                    (1.75, -8), (1.76, -7), (2.0, -7), (1e30, 56), (1e-30, -56),
                                    (448.0 * 2.0 ** 56, 56)])
def test_reference_exponent(amax, e):
    assert ref.exponent(np.array([0.0, -amax, np.inf, np.nan])) == e


def test_reference_write_and_read_round_trip():
    # values that E4M3 holds at the block's scale come back exactly, and a
    # growing scale keeps the earlier tokens
    codes, scales = np.zeros((2, 16, 1, 64), np.uint8), np.zeros((2, 1), np.uint8)
    x = np.zeros((3, 1, 64))
    x[0], x[1], x[2] = 1.0, -1.5, 3.0 * 2 ** 12
    bt = np.array([[1]])
    ref.write_one(x[:2], codes, scales, bt, [0, 2], [2])
    assert scales[1, 0] == 127 - 8
    ref.write_one(x[2:], codes, scales, bt, [0, 1], [3])
    assert scales[1, 0] == 127 + 12 - 7
    np.testing.assert_array_equal(ref.context(codes, scales, bt[0], 3), x)


def test_reference_attention_matches_dense():
    rng = np.random.default_rng(1)
    bt, nb = ref.tables(rng, [37])
    kc, ks = ref.make_pools(rng, nb, 2, 64)
    vc, vs = ref.make_pools(rng, nb, 2, 64)
    q = rng.standard_normal((5, 4, 64))
    out, mean, *_ = ref.attention(q, kc, vc, ks, vs, bt, [0, 5], [37], 0.125)
    want = dense_causal_numpy(q, ref.context(kc, ks, bt[0], 37), ref.context(vc, vs, bt[0], 37),
                              32, 0.125)
    np.testing.assert_allclose(out, want, rtol=1e-12, atol=1e-12)
    assert (np.abs(out) <= mean * (1 + 1e-12)).all()


def _write(**kw):
    a = dict(key=FAKE, value=FAKE, stride=256, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, mb=4,
             qsl=FAKE, sl=FAKE, r=2, t=3, h=2, d=128, bs=16, nb=8, dt=pa.PA_BF16)
    assert kw.keys() <= a.keys()
    a.update(kw)
    return pa.lib().pa_cache_write_scaled(
        a["key"], a["value"], a["stride"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["mb"],
        a["qsl"], a["sl"], a["r"], a["t"], a["h"], a["d"], a["bs"], a["nb"], a["dt"], None)


@pytest.mark.parametrize("kw", [dict(r=-1), dict(t=-1), dict(h=0), dict(d=0), dict(bs=0),
                                dict(nb=-1), dict(mb=-1), dict(dt=pa.PA_FP8_E4M3), dict(dt=9),
                                dict(stride=255), dict(nb=1 << 27), dict(key=None),
                                dict(value=None), dict(kc=None), dict(vc=None), dict(ks=None),
                                dict(vs=None), dict(bt=None), dict(qsl=None), dict(sl=None)])
def test_write_rejects_bad_arguments(kw):
    assert _write(**kw) == pa.PA_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(d=96, stride=192), dict(d=256, stride=512), dict(bs=32),
                                dict(stride=260), dict(key=ODD), dict(value=ODD), dict(kc=ODD),
                                dict(vc=ODD), dict(r=50_001)])
def test_write_refuses_unsupported(kw):
    assert _write(**kw) == pa.PA_ERR_UNSUPPORTED


def test_nothing_to_do_launches_nothing():
    assert _write(t=0, key=None, value=None) == pa.PA_OK
    assert _write(r=0, bt=None, qsl=None, sl=None) == pa.PA_OK
    assert _read(n=0, ko=None, vo=None) == pa.PA_OK
    assert _read(r=0, bt=None, first=None, starts=None) == pa.PA_OK
    assert _copy(n=0, ks=None, src=None) == pa.PA_OK
    assert _attend(t=0, q=None, out=None, ks=None) == pa.PA_OK
    assert pa.pa_launch_count() == 0


def _read(**kw):
    a = dict(kc=FAKE, vc=FAKE, cdt=pa.PA_FP8_E4M3, k1=None, v1=None, ks=FAKE, vs=FAKE, bt=FAKE,
             mb=4, first=FAKE, starts=FAKE, r=2, n=5, h=2, d=128, bs=16, nb=8, ko=FAKE, vo=FAKE,
             dt=pa.PA_BF16)
    assert kw.keys() <= a.keys()
    a.update(kw)
    return pa.lib().pa_cache_read(
        a["kc"], a["vc"], a["cdt"], a["k1"], a["v1"], a["ks"], a["vs"], a["bt"], a["mb"],
        a["first"], a["starts"], a["r"], a["n"], a["h"], a["d"], a["bs"], a["nb"], a["ko"],
        a["vo"], a["dt"], None)


@pytest.mark.parametrize("kw", [dict(r=-1), dict(n=-1), dict(h=0), dict(d=0), dict(bs=0),
                                dict(nb=-1), dict(mb=-1), dict(dt=pa.PA_FP8_E4M3),
                                dict(cdt=pa.PA_FP16), dict(ks=None), dict(vs=None),
                                dict(k1=FAKE), dict(v1=FAKE), dict(cdt=pa.PA_BF16),
                                dict(nb=1 << 27), dict(kc=None), dict(vc=None), dict(bt=None),
                                dict(first=None), dict(starts=None), dict(ko=None), dict(vo=None)])
def test_read_rejects_bad_arguments(kw):
    assert _read(**kw) == pa.PA_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(d=96), dict(d=36, ks=None, vs=None), dict(ko=ODD),
                                dict(vo=ODD), dict(kc=ODD), dict(vc=ODD),
                                dict(kc=ctypes.c_void_p(0x100008), cdt=pa.PA_BF16, ks=None,
                                     vs=None)])
def test_read_refuses_unsupported(kw):
    assert _read(**kw) == pa.PA_ERR_UNSUPPORTED


def _copy(**kw):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, src=FAKE, dst=FAKE, n=3, bs=16, h=2, d=64, nb=8)
    assert kw.keys() <= a.keys()
    a.update(kw)
    return pa.lib().pa_copy_blocks_scaled(a["kc"], a["vc"], a["ks"], a["vs"], a["src"], a["dst"],
                                          a["n"], a["bs"], a["h"], a["d"], a["nb"], None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(ks=None), dict(vs=None), dict(src=None),
                                dict(dst=None), dict(kc=ODD), dict(h=0)])
def test_copy_rejects_bad_arguments(kw):
    assert _copy(**kw) == pa.PA_ERR_INVALID


def _attend(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, mb=4, qsl=FAKE, sl=FAKE, r=2,
             t=3, mq=2, ml=16, hq=4, h=2, d=64, bs=16, nb=8, dt=pa.PA_BF16, flags=0, out=FAKE,
             ws=None, wsb=0)
    assert kw.keys() <= a.keys()
    a.update(kw)
    return pa.lib().pa_attention_scaled(
        a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["mb"], a["qsl"], a["sl"], a["r"],
        a["t"], a["mq"], a["ml"], a["hq"], a["h"], a["d"], a["bs"], a["nb"], 0.125, a["dt"],
        a["flags"], a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", [dict(ks=None), dict(vs=None), dict(q=None), dict(out=None),
                                dict(r=-1), dict(flags=2), dict(dt=pa.PA_FP8_E4M3), dict(q=ODD),
                                dict(kc=ODD), dict(ws=ODD, wsb=512), dict(nb=0), dict(mb=0)])
def test_attention_rejects_bad_arguments(kw):
    assert _attend(**kw) == pa.PA_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(d=96), dict(bs=32), dict(hq=5), dict(nb=1 << 28)])
def test_attention_refuses_unsupported(kw):
    assert _attend(**kw) == pa.PA_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    z = torch.zeros
    i, u, b = torch.int32, torch.uint8, torch.bfloat16
    pools = (z(2, 16, 1, 64, dtype=u), z(2, 16, 1, 64, dtype=u), z(2, 1, dtype=u), z(2, 1, dtype=u))
    bt, qsl, sl = z(1, 2, dtype=i), z(2, dtype=i), z(1, dtype=i)
    x = z(1, 1, 64, dtype=b)
    with pytest.raises(TypeError):
        pa.pa_cache_write_scaled(x, x, *pools, bt, qsl, sl)
    with pytest.raises(TypeError):
        pa.pa_cache_read(*pools[:2], bt, sl, qsl, x, x)
    with pytest.raises(TypeError):
        pa.pa_attention_scaled(x, *pools, bt, qsl, sl, 1, 1, 1.0, x)
    with pytest.raises(TypeError):
        pa.pa_copy_blocks_scaled(*pools, sl, sl)
