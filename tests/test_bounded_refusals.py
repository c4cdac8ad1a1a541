"""Refusals of norm_rope_store, prefill_window, decode_scored and evict: every
check returns before a CUDA call, so these run on the CPU."""
import ctypes

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


def norm_rope(L, cache=None, q=P(0x10), qs=512, k=P(0x20), ks=256, v=P(0x30), vs=256, T=3, H=4,
              qw=0x40, kw=0x50, cs=0x60, maxp=10, rot=128, eps=1e-6, pos=P(0x70), slots=P(0x80),
              scores=None, out=P(0x90), params=True):
    c = cache or _cache()
    p = pa.NormRope(qw, kw, cs, maxp, rot, 0, eps)
    return L.pa_norm_rope_store(q, qs, k, ks, v, vs, ctypes.byref(p) if params else None, pos,
                                slots, T, H, ctypes.byref(c), scores, out, None)


@pytest.mark.parametrize("kw, want", [
    (dict(params=False), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(slots=None), 1), (dict(out=None), 1), (dict(pos=None), 1), (dict(cs=None), 1),
    (dict(T=-1), 2), (dict(H=0), 2), (dict(rot=-16), 2), (dict(rot=144), 2), (dict(rot=24), 4),
    (dict(maxp=0), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(qs=511), 2), (dict(qs=516), 2), (dict(ks=248), 2), (dict(vs=260), 2),
    (dict(q=P(0x18)), 7), (dict(k=P(0x24)), 7), (dict(out=P(0x98)), 7), (dict(qw=0x42), 7),
    (dict(kw=0x58), 7), (dict(cs=0x64), 7), (dict(scores=P(0x104)), 7),
    (dict(out=P(0x10), qs=1024), 2),  # in place needs contiguous q
    (dict(T=0, q=None, out=None), 0),
])
def test_norm_rope_arguments(L, kw, want):
    assert norm_rope(L, **kw) == want


def prefill(L, cache=None, q=P(0x10), bt=P(0x20), mb=4, cq=P(0x30), ck=P(0x40), B=2, H=4, T=8,
            scale=0.1, window=16, sinks=0, out=P(0x50)):
    c = cache or _cache()
    return L.pa_prefill_window(q, ctypes.byref(c), bt, mb, cq, ck, B, H, T, 0, scale, window,
                               sinks, out, None)


@pytest.mark.parametrize("kw, want", [
    (dict(window=0), 2), (dict(window=-3), 2), (dict(sinks=-1), 2), (dict(mb=0), 2),
    (dict(q=None), 1), (dict(bt=None), 1), (dict(cq=None), 1), (dict(ck=None), 1),
    (dict(out=None), 1), (dict(H=3), 2), (dict(H=6), 4), (dict(H=64), 4), (dict(scale=0.0), 2),
    (dict(scale=float("inf")), 2), (dict(q=P(0x14)), 7), (dict(B=0), 0), (dict(T=0), 0),
    (dict(T=-1), 2),
])
def test_prefill_window_arguments(L, kw, want):
    assert prefill(L, **kw) == want


def test_prefill_window_needs_bf16_and_head_dim_128(L):
    assert prefill(L, _cache(head_dim=64)) == 4
    assert prefill(L, _cache(dtype=pa.PA_KV_FP8_E4M3, k_scale=0x3000, v_scale=0x4000)) == 4


def scored(L, cache=None, q=P(0x10), bt=P(0x20), mb=4, cl=P(0x30), B=2, H=4, scale=0.1,
           scores=P(0x40), out=P(0x50)):
    c = cache or _cache()
    return L.pa_decode_scored(q, ctypes.byref(c), bt, mb, cl, 0, B, H, scale, scores, out, None, 0,
                              None)


@pytest.mark.parametrize("kw, want", [
    (dict(scores=None), 1), (dict(scores=P(0x44)), 7), (dict(q=None), 1), (dict(bt=None), 1),
    (dict(cl=None), 1), (dict(out=None), 1), (dict(B=-1), 2), (dict(B=0), 0), (dict(H=3), 2),
    (dict(H=18), 4), (dict(mb=0), 2), (dict(scale=float("nan")), 2), (dict(out=P(0x58)), 7),
])
def test_decode_scored_arguments(L, kw, want):
    assert scored(L, **kw) == want


def evict(L, cache=None, scores=P(0x10), bt=P(0x20), mb=4, cl=P(0x1000), B=2, budget=16, sinks=2,
          recent=4, kept=P(0x2000), new=P(0x3000)):
    c = cache or _cache()
    return L.pa_evict(ctypes.byref(c), scores, bt, mb, cl, 0, B, budget, sinks, recent, kept, new,
                      None)


@pytest.mark.parametrize("kw, want", [
    (dict(scores=None), 1), (dict(bt=None), 1), (dict(cl=None), 1), (dict(kept=None), 1),
    (dict(new=None), 1), (dict(budget=0), 2), (dict(sinks=-1), 2), (dict(recent=-1), 2),
    (dict(sinks=10, recent=7), 2), (dict(sinks=0x7fffffff, recent=0x7fffffff), 2),
    (dict(B=-1), 2), (dict(mb=0), 2), (dict(B=0), 0), (dict(B=70000, new=P(0x9000000)), 4),
    (dict(new=P(0x1000)), 2), (dict(new=P(0x1004)), 2),  # new_lens over context_lens
    (dict(scores=P(0x18)), 7), (dict(mb=(1 << 26) + 1), 4),
])
def test_evict_arguments(L, kw, want):
    assert evict(L, **kw) == want


@pytest.mark.parametrize("budget", [(1 << 30) + 1, 0x7fffffff - 4096, 0x7fffffff])
def test_evict_refuses_budgets_whose_rows_32_bits_cannot_step_over(L, budget):
    assert evict(L, budget=budget) == 4


@pytest.mark.parametrize("kw, want", BAD_CACHES)
def test_every_call_checks_the_cache(L, kw, want):
    for f in (norm_rope, prefill, scored, evict):
        assert f(L, _cache(**kw)) == want, f.__name__


def test_scored_workspace_size_is_zero_for_invalid_arguments(L):
    c = _cache(num_blocks=0)
    assert L.pa_decode_scored_workspace_size(ctypes.byref(c), 4, 8, 4, 0) == 0
    c = _cache()
    assert L.pa_decode_scored_workspace_size(ctypes.byref(c), 0, 8, 4, 0) == 0


# ------------------------------------------------------------------ the binding
def _t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _norm_rope_args():
    return dict(q=_t((3, 4, 128)), k=_t((3, 2, 128)), v=_t((3, 2, 128)),
                positions=_t(3, torch.int64), slot_mapping=_t(3, torch.int64),
                k_cache=_t((8, 16, 2, 128)), v_cache=_t((8, 16, 2, 128)),
                cos_sin=_t((10, 128), torch.float32))


@pytest.mark.parametrize("kw, err", [
    (dict(q=_t((3, 4, 128), torch.float16)), TypeError), (dict(q=_t((3, 512))), ValueError),
    (dict(k=_t((3, 1, 128))), ValueError), (dict(v=_t((2, 2, 128))), ValueError),
    (dict(positions=_t(3, torch.int32)), TypeError), (dict(positions=None), ValueError),
    (dict(slot_mapping=_t(2, torch.int64)), ValueError),
    (dict(cos_sin=_t((10, 128), torch.float64)), TypeError), (dict(cos_sin=_t(128)), ValueError),
    (dict(q_weight=_t(64)), ValueError), (dict(k_weight=_t(128, torch.float32)), TypeError),
    (dict(q_out=_t((3, 4, 64))), ValueError), (dict(q_out=_t((4, 3, 128)).transpose(0, 1)), ValueError),
    (dict(scores=_t((8, 16, 2), torch.float32)), ValueError),
    (dict(v_cache=_t((8, 16, 2, 64))), ValueError), (dict(k_scale=_t((8, 2, 16), torch.float32)), ValueError),
    ({}, ValueError),  # CPU tensors
])
def test_norm_rope_binding(kw, err):
    a = _norm_rope_args()
    a.update(kw)
    args = [a.pop(n) for n in ("q", "k", "v", "positions", "slot_mapping", "k_cache", "v_cache")]
    with pytest.raises(err):
        pa.norm_rope_store(*args, **a)


def test_other_bindings_refuse_wrong_types_shapes_and_devices():
    kc, vc = _t((8, 16, 2, 128)), _t((8, 16, 2, 128))
    bt, cl = _t((2, 4), torch.int32), _t(2, torch.int32)
    cu, sc = _t(3, torch.int32), _t((8, 2, 16), torch.float32)
    q = _t((2, 4, 128))
    bad = [
        (pa.prefill_window, (q, kc, vc, bt, cu, cu, 0.1, 8), ValueError),  # CPU tensors
        (pa.prefill_window, (q.float(), kc, vc, bt, cu, cu, 0.1, 8), TypeError),
        (pa.prefill_window, (q, kc, vc, bt, cu.long(), cu, 0.1, 8), TypeError),
        (pa.prefill_window, (q, kc, vc, bt, cu, cu[:2], 0.1, 8), ValueError),
        (pa.prefill_window, (q, kc, vc, bt[:1], cu, cu, 0.1, 8), ValueError),
        (pa.decode_scored, (q, kc, vc, bt, cl, sc, 0.1), ValueError),
        (pa.decode_scored, (q, kc, vc, bt, cl, sc.half(), 0.1), TypeError),
        (pa.decode_scored, (q, kc, vc, bt, cl[:1], sc, 0.1), ValueError),
        (pa.decode_scored, (q, kc, vc, bt.long(), cl, sc, 0.1), TypeError),
        (pa.decode_scored, (q[0], kc, vc, bt, cl, sc, 0.1), ValueError),
        (pa.decode_scored, (q, kc, vc, bt, cl, sc.transpose(1, 2), 0.1), ValueError),
        (pa.evict, (kc, vc, sc, bt, cl, 16), ValueError),
        (pa.evict, (kc, vc, sc, bt, cl.long(), 16), TypeError),
        (pa.evict, (kc, vc, sc, bt[0], cl, 16), ValueError),
        (pa.evict, (kc, vc[:4], sc, bt, cl, 16), ValueError),
    ]
    for fn, args, err in bad:
        with pytest.raises(err):
            fn(*args)


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63, -2 ** 32 + 5])
def test_bindings_refuse_numbers_that_do_not_fit_32_bits(big):
    # ctypes drops their upper bits: a window of 2^32 + 1 would be a window of 1
    kc, vc = _t((8, 16, 2, 128)), _t((8, 16, 2, 128))
    bt, cl = _t((2, 4), torch.int32), _t(2, torch.int32)
    cu, sc = _t(3, torch.int32), _t((8, 2, 16), torch.float32)
    q = _t((2, 4, 128))
    calls = [
        (pa.prefill_window, (q, kc, vc, bt, cu, cu, 0.1, big), {}, "window"),
        (pa.prefill_window, (q, kc, vc, bt, cu, cu, 0.1, 8, big), {}, "sinks"),
        (pa.prefill_window, (q, kc, vc, bt, cu, cu, 0.1, 8), dict(max_q_len=big), "max_q_len"),
        (pa.decode_scored, (q, kc, vc, bt, cl, sc, 0.1), dict(max_context_len=big),
         "max_context_len"),
        (pa.decode_scored_workspace_size, (kc, 2, 4, 4), dict(max_context_len=big),
         "max_context_len"),
        (pa.decode_scored_workspace_size, (kc, big, 4, 4), {}, "batch"),
        (pa.evict, (kc, vc, sc, bt, cl, big), {}, "budget"),
        (pa.evict, (kc, vc, sc, bt, cl, 16), dict(sinks=big), "sinks"),
        (pa.evict, (kc, vc, sc, bt, cl, 16), dict(recent=big), "recent"),
        (pa.evict, (kc, vc, sc, bt, cl, 16), dict(max_context_len=big), "max_context_len"),
    ]
    for fn, args, kw, name in calls:
        with pytest.raises(ValueError, match=f"{name} must fit 32 bits"):
            fn(*args, **kw)
