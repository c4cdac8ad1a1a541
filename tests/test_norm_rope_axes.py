"""pa_norm_rope_axes_store against a plain 64-bit implementation.

Bounds as in test_norm_rope.py: the arithmetic of a row is the same, only the
table entries of a pair come from the row of the pair's own axis.
"""
import numpy as np
import pytest
import torch

import ops64
import paged_kv_cache_186_gb300 as pa
from test_norm_rope import EPS, FP32, check_rows, make

pytestmark = pytest.mark.gpu


def axes_inputs(T, H, Hkv, D, bs, kv="bf16", rot=None, axes=3, layout="sections", seed=0, **kw):
    s = make(T, H, Hkv, D, bs, kv, rot, seed=seed, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    half = s["rot"] // 2
    s["axes"] = axes
    s["pos"] = torch.randint(0, s["cs"].shape[0], (axes, T), generator=g).cuda()
    if layout == "sections":
        s["map"] = [i * axes // half for i in range(half)]
    elif layout == "cycle":
        s["map"] = [i % axes for i in range(half)]
    else:
        s["map"] = torch.randint(0, axes, (half,), generator=g).tolist()
    return s


def call(s, interleaved=False, scores=True, weights=True, **kw):
    out = pa.norm_rope_axes_store(
        s["q"], s["k"], s["v"], s["pos"], s["slots"], s["kc"], s["vc"], s["map"], s["cs"],
        q_weight=s["qw"] if weights else None, k_weight=s["kw"] if weights else None, eps=EPS,
        interleaved=interleaved, k_scale=s["ks"], v_scale=s["vs"],
        scores=s["scores"] if scores else None, **kw)
    torch.cuda.synchronize()
    return out


def n64(t):
    return t.float().cpu().double().numpy()


def want64(s, x, weight, interleaved):
    """(y, magnitude) of ops64.norm_rope with every pair's own row of the table."""
    pos, cs = s["pos"].cpu().numpy(), s["cs"].cpu().numpy()
    half = s["rot"] // 2
    rows = np.empty((x.shape[0], s["rot"]), dtype=np.float32)  # each token's own table row
    for i, a in enumerate(s["map"]):
        rows[:, i], rows[:, half + i] = cs[pos[a], i], cs[pos[a], half + i]
    return ops64.norm_rope(n64(x), weight, EPS, rows, np.arange(x.shape[0]), interleaved)


def check(s, before, out, interleaved=False, weights=True, live=None):
    slots = s["slots"].cpu().numpy()
    live = slots >= 0 if live is None else live
    q, qm = want64(s, s["q"], n64(s["qw"]) if weights else None, interleaved)
    k, km = want64(s, s["k"], n64(s["kw"]) if weights else None, interleaved)
    check_rows(n64(out)[live], q[live], qm[live], "q_out")
    b, o = slots[live] // s["bs"], slots[live] % s["bs"]
    v = n64(s["v"])
    for x, m, cache, scale in ((k[live], km[live], "kc", "ks"),
                               (v[live], np.abs(v[live]), "vc", "vs")):
        new, old = s[cache].cpu(), before[cache].cpu()
        if s["kv"] == "bf16":
            check_rows(n64(new)[b, o], x, m, cache)
        else:
            top = ops64.FP8_MAX if s["kv"] == "fp8" else ops64.INT8_MAX
            sc = s[scale].cpu().double().numpy()[b, :, o]
            want = np.abs(x).max(-1) / top
            assert (np.abs(sc - want) <= m.max(-1) * FP32 / top + want * 2.0 ** -23).all()
            got = ops64.cache_values(new, s[scale].cpu())[b, o]
            step = (np.maximum(np.abs(x) * 2.0 ** -4, sc[..., None] * 2.0 ** -10)
                    if s["kv"] == "fp8" else sc[..., None] * 0.5)
            tol = step * (1 + 2.0 ** -20) + 3 * m.max(-1, keepdims=True) * FP32
            assert (np.abs(got - x) <= tol).all(), cache
        mask = np.ones(tuple(new.shape[:2]), bool)
        mask[b, o] = False
        view = (lambda t: t.view(torch.int16)) if s["kv"] == "bf16" else (lambda t: t)
        assert torch.equal(view(new)[torch.from_numpy(mask)], view(old)[torch.from_numpy(mask)])
    sc = s["scores"].cpu()
    assert (sc[b, :, o] == 0).all()


def copies(s):
    return {n: s[n].clone() for n in ("kc", "vc", "scores")}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout", ["sections", "cycle", "random"])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("D, rot, kv", [(128, 128, "bf16"), (64, 64, "bf16"), (128, 64, "fp8"),
                                        (64, 48, "bf16"), (128, 112, "int8")])
def test_matches_64_bits(D, rot, kv, axes, layout, interleaved):
    s = axes_inputs(37, 6, 2, D, 16, kv, rot, axes, layout, seed=axes + rot)
    s["slots"][5] = -1
    before = copies(s)
    out0 = torch.full_like(s["q"], 7.0).contiguous()
    out = call(s, interleaved, q_out=out0)
    assert pa.get_device_error() == 0
    check(s, before, out, interleaved)
    assert (out[5] == 7.0).all()


@pytest.mark.parametrize("T, H, Hkv, D, kv", [(1, 1, 1, 64, "bf16"), (1, 32, 8, 128, "fp8"),
                                              (700, 32, 8, 128, "bf16"), (3001, 16, 4, 128, "int8"),
                                              (2500, 24, 8, 64, "bf16"), (1500, 40, 8, 128, "fp8")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_every_launch_form(T, H, Hkv, D, kv, interleaved):
    s = axes_inputs(T, H, Hkv, D, 32, kv, D, 3, "random", seed=T)
    before = copies(s)
    check(s, before, call(s, interleaved), interleaved)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("T", [3, 2000])
def test_one_axis_and_equal_axes_are_norm_rope_store(kv, T):
    s = axes_inputs(T, 8, 2, 128, 16, kv, 128, 1, seed=9)
    plain = dict(s, kc=s["kc"].clone(), vc=s["vc"].clone())
    if kv != "bf16":
        plain["ks"], plain["vs"] = s["ks"].clone(), s["vs"].clone()
    want = pa.norm_rope_store(plain["q"], plain["k"], plain["v"], s["pos"][0], plain["slots"],
                              plain["kc"], plain["vc"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                              cos_sin=s["cs"], k_scale=plain["ks"], v_scale=plain["vs"])
    first = s["pos"]
    for axes in (1, 4):
        s["pos"] = first.expand(axes, T)  # (a stride of 0 between the axes)
        s["map"] = [i % axes for i in range(64)]
        out = call(s, scores=False)
        assert torch.equal(out, want)
        assert torch.equal(s["kc"], plain["kc"]) and torch.equal(s["vc"], plain["vc"])
        if kv != "bf16":
            assert torch.equal(s["ks"], plain["ks"]) and torch.equal(s["vs"], plain["vs"])


def test_without_weights_and_in_place():
    s = axes_inputs(50, 8, 2, 128, 16, fused=False, seed=11)
    before = copies(s)
    q = s["q"].clone()
    s2 = dict(s, q=q)
    out = call(s2, weights=False, q_out=q)
    assert out is q
    check(s, before, out, weights=False)


@pytest.mark.parametrize("axis", [0, 1, 2])
@pytest.mark.parametrize("bad", [-1, 512, 1 << 40, -(1 << 62)])
def test_a_position_outside_the_table_on_any_axis_skips_the_token(axis, bad):
    s = axes_inputs(20, 8, 2, 128, 16, seed=12)
    s["map"] = [i % 2 for i in range(64)]  # the third axis turns no pair and is checked all the same
    s["pos"][axis, 4] = bad
    before = copies(s)
    q_out = torch.full((20, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    out = call(s, q_out=q_out)
    assert pa.get_device_error() == pa.PA_DEVERR_POSITION_RANGE
    assert (out[4] == 5.0).all()
    s["pos"][axis, 4] = 0
    live = np.arange(20) != 4
    check(s, before, out, live=live)
    slot = s["slots"][4].item()
    assert torch.equal(s["kc"][slot // 16, slot % 16], before["kc"][slot // 16, slot % 16])


def test_out_of_range_slots_are_flagged():
    s = axes_inputs(9, 4, 2, 64, 16, seed=13)
    s["slots"][2] = s["kc"].shape[0] * 16
    before = copies(s)
    call(s)
    assert pa.get_device_error() == pa.PA_DEVERR_SLOT_RANGE
    live = np.arange(9) != 2
    slot = s["slots"].cpu().numpy()[live]
    mask = np.ones((s["kc"].shape[0], 16), bool)
    mask[slot // 16, slot % 16] = False
    assert torch.equal(s["kc"].cpu()[torch.from_numpy(mask)], before["kc"].cpu()[torch.from_numpy(mask)])


def test_captured_and_on_another_stream():
    s = axes_inputs(33, 8, 2, 128, 16, seed=14)
    before = copies(s)
    out = torch.zeros((33, 8, 128), dtype=torch.bfloat16, device="cuda")
    call(s, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.norm_rope_axes_store(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["kc"], s["vc"],
                                s["map"], s["cs"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                q_out=out, scores=s["scores"])
    s["pos"].copy_(torch.randint(0, 512, (3, 33)))
    graph.replay()
    torch.cuda.synchronize()
    check(s, before, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = pa.norm_rope_axes_store(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["kc"],
                                        s["vc"], bytes(s["map"]), s["cs"], q_weight=s["qw"],
                                        k_weight=s["kw"], eps=EPS)
    side.synchronize()
    assert torch.equal(other, out)


def test_no_tokens():
    s = axes_inputs(1, 8, 2, 128, 16, seed=15)
    out = pa.norm_rope_axes_store(s["q"][:0], s["k"][:0], s["v"][:0], s["pos"][:, :0],
                                  s["slots"][:0], s["kc"], s["vc"], s["map"], s["cs"])
    assert out.shape == (0, 8, 128)
