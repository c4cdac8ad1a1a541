"""Refusals of norm_rope_axes_store, decode_shared and prefill_shared: every check returns before
a CUDA call, so these run on the CPU."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_186_gb300 as pa
from paged_kv_cache_186_gb300 import build as pabuild

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    pabuild.build()
    return pa.lib()


def _cache(**kw):
    c = dict(num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128, dtype=pa.PA_KV_BF16,
             k_cache=0x1000, v_cache=0x2000, k_scale=None, v_scale=None)
    c.update(kw)
    return pa.KVCache(**c)


BAD_CACHES = [(dict(k_cache=None), 1), (dict(num_blocks=0), 2), (dict(dtype=7), 3),
              (dict(dtype=pa.PA_KV_FP8_E4M3), 3), (dict(k_scale=0x3000, v_scale=0x4000), 3),
              (dict(block_size=8), 4), (dict(head_dim=96), 4), (dict(v_cache=0x1004), 7)]


def axes(L, cache=None, q=P(0x10), qs=512, k=P(0x20), ks=256, v=P(0x30), vs=256, T=3, H=4,
         qw=0x40, kw=0x50, cs=0x60, maxp=10, rot=128, eps=1e-6, pos=P(0x70), n=3,
         pair=bytes([0] * 16 + [1] * 24 + [2] * 24), slots=P(0x80), scores=None, out=P(0x90),
         params=True):
    c = cache or _cache()
    p = pa.NormRope(qw, kw, cs, maxp, rot, 0, eps)
    return L.pa_norm_rope_axes_store(q, qs, k, ks, v, vs, ctypes.byref(p) if params else None, pos,
                                     n, pair, slots, T, H, ctypes.byref(c), scores, out, None)


@pytest.mark.parametrize("kw, want", [
    (dict(params=False), 1), (dict(pair=None), 1), (dict(pos=None), 1), (dict(cs=None), 1),
    (dict(q=None), 1), (dict(slots=None), 1), (dict(out=None), 1),
    (dict(n=0), 2), (dict(n=-1), 2), (dict(n=2), 2), (dict(n=5), 4),
    (dict(pair=bytes([3] * 64)), 2), (dict(pair=bytes([0] * 63 + [255])), 2),
    (dict(rot=0), 2), (dict(rot=-16), 2), (dict(rot=144), 2), (dict(rot=24), 4), (dict(maxp=0), 2),
    (dict(eps=-1.0), 2), (dict(qs=511), 2), (dict(T=-1), 2), (dict(H=0), 2),
    (dict(q=P(0x18)), 7), (dict(cs=0x64), 7), (dict(scores=P(0x104)), 7),
    (dict(out=P(0x10), qs=1024), 2), (dict(T=0, q=None, out=None), 0),
])
def test_norm_rope_axes_arguments(L, kw, want):
    assert axes(L, **kw) == want


def decode(L, cache=None, q=P(0x10), bt=P(0x20), mb=4, cl=P(0x30), cu=P(0x40), pl=P(0x50), G=1,
           B=2, H=4, scale=0.1, out=P(0x60)):
    c = cache or _cache()
    return L.pa_decode_shared(q, ctypes.byref(c), bt, mb, cl, 0, cu, pl, G, 0, B, H, scale, out,
                              None, 0, None)


@pytest.mark.parametrize("kw, want", [
    (dict(q=None), 1), (dict(bt=None), 1), (dict(cl=None), 1), (dict(out=None), 1),
    (dict(cu=None), 1), (dict(pl=None), 1), (dict(G=-1), 2), (dict(B=-1), 2), (dict(mb=0), 2),
    (dict(H=3), 2), (dict(H=18), 4), (dict(B=16385), 4), (dict(G=16385), 4),
    (dict(scale=float("nan")), 2), (dict(scale=0.0), 2), (dict(scale=-0.1), 2),
    (dict(q=P(0x18)), 7), (dict(out=P(0x68)), 7), (dict(B=0), 0),
    (dict(B=0, G=0, cu=None, pl=None), 0),
])
def test_decode_shared_arguments(L, kw, want):
    assert decode(L, **kw) == want


def prefill(L, cache=None, q=P(0x10), bt=P(0x20), mb=4, cq=P(0x30), ck=P(0x40), cu=P(0x50),
            pl=P(0x60), G=1, B=2, H=4, T=8, scale=0.1, out=P(0x70)):
    c = cache or _cache()
    return L.pa_prefill_shared(q, ctypes.byref(c), bt, mb, cq, ck, cu, pl, G, 0, B, H, T, 0, scale,
                               out, None, 0, None)


@pytest.mark.parametrize("kw, want", [
    (dict(q=None), 1), (dict(bt=None), 1), (dict(cq=None), 1), (dict(ck=None), 1),
    (dict(out=None), 1), (dict(cu=None), 1), (dict(pl=None), 1), (dict(G=-1), 2), (dict(mb=0), 2),
    (dict(B=-1), 2), (dict(T=-1), 2), (dict(H=3), 2), (dict(H=6), 4), (dict(H=64), 4),
    (dict(B=16385), 4), (dict(G=16385), 4), (dict(scale=0.0), 2), (dict(scale=float("inf")), 2),
    (dict(q=P(0x14)), 7), (dict(B=0), 0), (dict(T=0), 0),
])
def test_prefill_shared_arguments(L, kw, want):
    assert prefill(L, **kw) == want


def test_prefill_shared_needs_bf16_and_head_dim_128(L):
    assert prefill(L, _cache(head_dim=64)) == 4
    assert prefill(L, _cache(dtype=pa.PA_KV_FP8_E4M3, k_scale=0x3000, v_scale=0x4000)) == 4


@pytest.mark.parametrize("kw, want", BAD_CACHES)
def test_every_call_checks_the_cache(L, kw, want):
    for f in (axes, decode, prefill):
        assert f(L, _cache(**kw)) == want, f.__name__


def test_workspace_sizes_are_zero_for_invalid_arguments(L):
    bad, c = _cache(num_blocks=0), _cache()
    d, p = L.pa_decode_shared_workspace_size, L.pa_prefill_shared_workspace_size
    assert d(ctypes.byref(bad), 4, 8, 4, 1, 0) == 0 and p(ctypes.byref(bad), 8, 4, 1) == 0
    assert d(ctypes.byref(c), 0, 8, 4, 1, 0) == 0 and d(ctypes.byref(c), 4, 8, 4, -1, 0) == 0
    assert d(ctypes.byref(c), 16385, 8, 4, 1, 0) == 0 and d(ctypes.byref(c), 4, 8, 4, 16385, 0) == 0
    assert p(ctypes.byref(c), 0, 4, 1) == 0 and p(ctypes.byref(c), 8, 0, 1) == 0
    assert p(ctypes.byref(c), 8, 4, -1) == 0 and p(ctypes.byref(c), 8, 4, 16385) == 0


# ------------------------------------------------------------------ the binding
def _t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw, err", [
    (dict(q=_t((3, 4, 128), torch.float16)), TypeError), (dict(q=_t((3, 512))), ValueError),
    (dict(positions=_t(3, torch.int64)), ValueError), (dict(positions=None), ValueError),
    (dict(positions=_t((3, 2), torch.int64)), ValueError),
    (dict(positions=_t((3, 3), torch.int32)), TypeError), (dict(cos_sin=None), ValueError),
    (dict(pair_axis=[0] * 63), ValueError), (dict(pair_axis=[0] * 63 + [256]), ValueError),
    (dict(pair_axis=[0] * 63 + [-1]), ValueError), (dict(pair_axis=[0.5] * 64), TypeError),
    (dict(slot_mapping=_t(2, torch.int64)), ValueError),
    (dict(cos_sin=_t((10, 128), torch.float64)), TypeError),
    ({}, ValueError),  # CPU tensors
])
def test_norm_rope_axes_binding(kw, err):
    a = dict(q=_t((3, 4, 128)), k=_t((3, 2, 128)), v=_t((3, 2, 128)),
             positions=_t((3, 3), torch.int64), slot_mapping=_t(3, torch.int64),
             k_cache=_t((8, 16, 2, 128)), v_cache=_t((8, 16, 2, 128)), pair_axis=bytes(64),
             cos_sin=_t((10, 128), torch.float32))
    a.update(kw)
    with pytest.raises(err):
        pa.norm_rope_axes_store(*a.values())


def test_shared_bindings_refuse_wrong_types_shapes_and_devices():
    kc, vc = _t((8, 16, 2, 128)), _t((8, 16, 2, 128))
    bt, cl = _t((2, 4), torch.int32), _t(2, torch.int32)
    cu, cg, pl = _t(3, torch.int32), _t(2, torch.int32), _t(1, torch.int32)
    q = _t((2, 4, 128))
    d, p = pa.decode_shared, pa.prefill_shared
    bad = [
        (d, (q, kc, vc, bt, cl, cg, pl, 0.1), ValueError),  # CPU tensors
        (d, (q.float(), kc, vc, bt, cl, cg, pl, 0.1), TypeError),
        (d, (q, kc, vc, bt.long(), cl, cg, pl, 0.1), TypeError),
        (d, (q, kc, vc, bt, cl[:1], cg, pl, 0.1), ValueError),
        (d, (q, kc, vc, bt, cl, cg[:1], pl, 0.1), ValueError),
        (d, (q, kc, vc, bt, cl, cg.long(), pl, 0.1), TypeError),
        (d, (q, kc, vc, bt, cl, cg, pl.float(), 0.1), TypeError),
        (d, (q[0], kc, vc, bt, cl, cg, pl, 0.1), ValueError),
        (d, (q, kc, vc[:4], bt, cl, cg, pl, 0.1), ValueError),
        (p, (q, kc, vc, bt, cu, cu, cg, pl, 0.1), ValueError),
        (p, (q.float(), kc, vc, bt, cu, cu, cg, pl, 0.1), TypeError),
        (p, (q, kc, vc, bt, cu.long(), cu, cg, pl, 0.1), TypeError),
        (p, (q, kc, vc, bt, cu, cu[:2], cg, pl, 0.1), ValueError),
        (p, (q, kc, vc, bt[:1], cu, cu, cg, pl, 0.1), ValueError),
        (p, (q, kc, vc, bt, cu, cu, cu, pl, 0.1), ValueError),
        (p, (q[0], kc, vc, bt, cu, cu, cg, pl, 0.1), ValueError),
    ]
    for fn, args, err in bad:
        with pytest.raises(err):
            fn(*args)


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63, -2 ** 32 + 5])
def test_shared_bindings_refuse_numbers_that_do_not_fit_32_bits(big):
    kc, vc = _t((8, 16, 2, 128)), _t((8, 16, 2, 128))
    bt, cl = _t((2, 4), torch.int32), _t(2, torch.int32)
    cu, cg, pl = _t(3, torch.int32), _t(2, torch.int32), _t(1, torch.int32)
    q = _t((2, 4, 128))
    calls = [
        (pa.decode_shared, (q, kc, vc, bt, cl, cg, pl, 0.1), dict(max_context_len=big),
         "max_context_len"),
        (pa.decode_shared_workspace_size, (kc, 2, 4, 4, big), {}, "num_groups"),
        (pa.decode_shared_workspace_size, (kc, big, 4, 4, 1), {}, "batch"),
        (pa.prefill_shared, (q, kc, vc, bt, cu, cu, cg, pl, 0.1), dict(max_q_len=big), "max_q_len"),
        (pa.prefill_shared_workspace_size, (kc, big, 4, 1), {}, "total_q"),
    ]
    for fn, args, kw, name in calls:
        with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
            fn(*args, **kw)


@pytest.mark.parametrize("pair_axis", [64, torch.tensor(64), np.int64(64), "axes", None,
                                       np.arange(8), np.zeros(64), torch.zeros(64)])
def test_axes_that_are_not_integers_one_a_pair_are_refused(pair_axis):
    # (64 is no list of 64 zeros, and 8 numbers of 8 bytes are not 64 axes)
    with pytest.raises((TypeError, ValueError)) as e:
        _axes_call(pair_axis)
    assert "caches' device" not in str(e.value) and "CUDA" not in str(e.value)


@pytest.mark.parametrize("pair_axis", [[0, 1] * 32, (0, 1) * 32, bytes([0, 1] * 32),
                                       bytearray([0, 1] * 32), np.arange(64) % 2,
                                       (np.arange(64) % 2).astype(np.int32), torch.arange(64) % 2])
def test_axes_of_any_integers_reach_the_call(pair_axis, monkeypatch):
    seen = []
    monkeypatch.setattr(pa, "_norm_rope", lambda *a: seen.append(a[7]))
    _axes_call(pair_axis)
    assert seen == [bytes([0, 1] * 32)]


def _axes_call(pair_axis):
    pa.norm_rope_axes_store(_t((3, 4, 128)), _t((3, 2, 128)), _t((3, 2, 128)),
                            _t((2, 3), torch.int64), _t(3, torch.int64), _t((8, 16, 2, 128)),
                            _t((8, 16, 2, 128)), pair_axis, _t((10, 128), torch.float32))
