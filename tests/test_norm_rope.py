"""pa_norm_rope_store against a plain 64-bit implementation.

Bounds. q_out and bf16 cache rows are one rounding to bf16 (at most 2^-8 of the
value) of an fp32 result y = rstd * (x A + x' B). Each of A, B, the products, the
fused add and the last product rounds once (2^-24 relative each), the mean of
the squares (8 fused adds, up to 4 shuffle adds, a product, an add) at most 14
times - 7 in rstd after the square root - and rsqrtf adds at most 2 ulp
(4 * 2^-24): together at most 16 * 2^-24 of rstd * (|x A| + |x' B|). The tests
allow 2^-19 of that magnitude (32 * 2^-24).
8-bit codes are one rounding of x / s: at most 2^-4 of the value or half the
smallest step (2^-10 s) for E4M3, half a step (s / 2) for INT8, next to the
fp32 error above; s itself carries the fp32 error of max|x| and two roundings.
"""
import numpy as np
import pytest
import torch

import ops64
import paged_kv_cache_186_gb300 as pa

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -19  # of the magnitude (see above)
EPS = 1e-6


def table(max_pos, rot, base=10000.0):
    half = rot // 2
    ang = np.arange(max_pos, dtype=np.float64)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def make(T, H, Hkv, D, bs, kv="bf16", rot=None, seed=0, max_pos=512, fused=True, pool=None):
    g = torch.Generator().manual_seed(seed)
    rot = D if rot is None else rot
    qkv = (torch.randn((T, (H + 2 * Hkv) * D), generator=g) * 3).to(torch.bfloat16).cuda()
    nb = pool or (T // bs + 3)
    s = dict(T=T, H=H, Hkv=Hkv, D=D, bs=bs, kv=kv, rot=rot)
    cut = [qkv[:, :H * D], qkv[:, H * D:(H + Hkv) * D], qkv[:, (H + Hkv) * D:]]
    s["q"], s["k"], s["v"] = (x.view(T, -1, D) if fused else x.reshape(T, -1, D).contiguous()
                              for x in cut)
    s["qw"], s["kw"] = (1 + 0.3 * torch.randn((2, D), generator=g)).to(torch.bfloat16).cuda()
    shape = (nb, bs, Hkv, D)
    if kv == "bf16":
        s["kc"], s["vc"] = (torch.randn(shape, generator=g).to(torch.bfloat16).cuda()
                            for _ in range(2))
        s["ks"] = s["vs"] = None
    else:
        dt = torch.uint8 if kv == "fp8" else torch.int8
        lo, hi = (0, 100) if kv == "fp8" else (-127, 128)
        s["kc"], s["vc"] = (torch.randint(lo, hi, shape, generator=g).to(dt).cuda()
                            for _ in range(2))
        s["ks"], s["vs"] = (torch.rand((nb, Hkv, bs), generator=g).cuda() for _ in range(2))
    s["slots"] = torch.randperm(nb * bs, generator=g)[:T].cuda()
    s["pos"] = torch.randint(0, max_pos, (T,), generator=g).cuda()
    s["cs"] = torch.from_numpy(table(max_pos, rot)).cuda() if rot else None
    s["scores"] = torch.rand((nb, Hkv, bs), generator=g).cuda()
    return s


def call(s, interleaved=False, q_weight=True, k_weight=True, scores=True, **kw):
    out = pa.norm_rope_store(
        s["q"], s["k"], s["v"], s["pos"], s["slots"], s["kc"], s["vc"],
        q_weight=s["qw"] if q_weight else None, k_weight=s["kw"] if k_weight else None, eps=EPS,
        cos_sin=s["cs"], interleaved=interleaved, k_scale=s["ks"], v_scale=s["vs"],
        scores=s["scores"] if scores else None, **kw)
    torch.cuda.synchronize()
    return out


def check_rows(got, want, mag, what):
    err = np.abs(got - want)
    tol = np.abs(want) * 2.0 ** -8 + mag * FP32
    assert (err <= tol).all(), f"{what}: {float((err - tol).max()):.3e} past the bound"


def check(s, before, out, interleaved=False, q_weight=True, k_weight=True):
    """Everything the call may write against the 64-bit implementation, everything else
    against what it was."""
    n64 = lambda t: t.float().cpu().double().numpy()
    slots = s["slots"].cpu().numpy()
    pos = s["pos"].cpu().numpy()
    cs = None if s["cs"] is None else s["cs"].cpu().numpy()
    live = slots >= 0
    q, qm = ops64.norm_rope(n64(s["q"]), n64(s["qw"]) if q_weight else None, EPS, cs, pos,
                            interleaved)
    k, km = ops64.norm_rope(n64(s["k"]), n64(s["kw"]) if k_weight else None, EPS, cs, pos,
                            interleaved)
    check_rows(n64(out)[live], q[live], qm[live], "q_out")
    v = n64(s["v"])
    b, o = slots[live] // s["bs"], slots[live] % s["bs"]
    for x, m, cache, scale, name in ((k, km, "kc", "ks", "k"), (v, np.abs(v), "vc", "vs", "v")):
        x, m = x[live], m[live]
        new, old = s[cache].cpu(), before[cache].cpu()
        if s["kv"] == "bf16":
            check_rows(n64(new)[b, o], x, m, name)
            if name == "v":
                assert np.array_equal(n64(new)[b, o], x)
        else:
            top = ops64.FP8_MAX if s["kv"] == "fp8" else ops64.INT8_MAX
            sc = s[scale].cpu().double().numpy()[b, :, o]
            want = np.abs(x).max(-1) / top
            want[want == 0] = 1.0
            # |x| is off by FP32 of its magnitude, the quotient rounds once
            stol = m.max(-1) * FP32 / top + want * 2.0 ** -23
            assert (np.abs(sc - want) <= stol).all(), name
            got = ops64.cache_values(new, s[scale].cpu())[b, o]
            step = (np.maximum(np.abs(x) * 2.0 ** -4, sc[..., None] * 2.0 ** -10)
                    if s["kv"] == "fp8" else sc[..., None] * 0.5)
            # the fp32 error of x and of x / s, and s's own error, move the value by
            # no more than three times FP32 of the largest magnitude of the row
            tol = step * (1 + 2.0 ** -20) + 3 * m.max(-1, keepdims=True) * FP32
            assert (np.abs(got - x) <= tol).all(), name
            # scales elsewhere
            mask = np.ones(s[scale].shape, bool)
            mask[b, :, o] = False
            assert torch.equal(s[scale].cpu()[torch.from_numpy(mask)],
                               before[scale].cpu()[torch.from_numpy(mask)])
        mask = np.ones(tuple(new.shape[:2]), bool)
        mask[b, o] = False
        raw = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t
        assert torch.equal(raw(new)[torch.from_numpy(mask)], raw(old)[torch.from_numpy(mask)])
    sc, old = s["scores"].cpu().numpy(), before["scores"].cpu().numpy().copy()
    old[b, :, o] = 0.0
    assert np.array_equal(sc, old)


def snapshot(s):
    return {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in s.items()}


CASES = [
    # T, H, Hkv, D, bs, kv, rot, interleaved
    (1, 8, 2, 64, 16, "bf16", 64, False),
    (1, 1, 1, 128, 32, "bf16", 128, True),
    (37, 32, 8, 128, 16, "bf16", 128, False),
    (37, 32, 8, 128, 16, "bf16", 64, True),
    (19, 5, 1, 128, 16, "bf16", 96, False),
    (19, 5, 3, 64, 32, "bf16", 48, False),
    (19, 5, 3, 64, 32, "bf16", 16, True),
    (11, 12, 4, 128, 32, "bf16", 0, False),
    (37, 64, 8, 128, 32, "fp8", 128, False),
    (13, 7, 7, 128, 16, "fp8", 32, True),
    (37, 40, 8, 128, 32, "int8", 128, False),
    (13, 6, 2, 128, 16, "int8", 112, False),
    (700, 32, 8, 128, 16, "bf16", 128, False),
    (701, 9, 3, 128, 16, "fp8", 128, True),
    (600, 16, 4, 128, 32, "int8", 64, False),
    (900, 33, 5, 64, 16, "bf16", 32, False),
    (300, 71, 2, 128, 16, "bf16", 128, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("weights", [(True, True), (False, True), (False, False)])
def test_matches_64_bits(case, weights):
    T, H, Hkv, D, bs, kv, rot, inter = case
    s = make(T, H, Hkv, D, bs, kv, rot, seed=T + H + D + rot)
    if T > 4:
        s["slots"][T // 2] = -1  # a padding token
    before = snapshot(s)
    out = call(s, inter, *weights)
    assert pa.get_device_error() == 0
    check(s, before, out, inter, *weights)


@pytest.mark.parametrize("T", [9000, 20011])
def test_large_batches(T):
    s = make(T, 8, 2, 128, 16, "bf16", 128, seed=T)
    before = snapshot(s)
    out = call(s)
    check(s, before, out)


def test_far_positions_use_their_own_row():
    s = make(16, 4, 2, 128, 16, seed=5, max_pos=131072)
    s["pos"][:] = torch.arange(131072 - 16, 131072)
    before = snapshot(s)
    check(s, before, call(s))


def test_v_codes_and_scales_are_the_plain_recipe_bit_for_bit():
    for kv, top in (("fp8", 448.0), ("int8", 127.0)):
        s = make(50, 2, 4, 128, 16, kv, seed=6)
        s["v"] = s["v"].clone()
        s["v"][3, 1] = 0.0                      # a row of zeros
        s["v"][4, 2] *= 2.0 ** -120             # a tiny row
        s["v"][5] *= 2.0 ** 110                 # large rows
        call(s)
        x = s["v"].float().cpu()
        amax = x.abs().amax(-1)
        sc = torch.where(amax > 0, amax / top, torch.ones_like(amax))
        y = x / sc[..., None]
        b, o = s["slots"].cpu() // 16, s["slots"].cpu() % 16
        assert torch.equal(s["vs"].cpu()[b, :, o], sc)
        want = (y.to(torch.float8_e4m3fn).view(torch.uint8) if kv == "fp8"
                else torch.round(y).clamp(-127, 127).to(torch.int8))
        assert torch.equal(s["vc"].cpu()[b, o], want)


@pytest.mark.parametrize("kv", ["fp8", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_with_a_nan_or_infinity_reads_back_as_nan(kv, bad):
    s = make(6, 2, 2, 128, 16, kv, seed=7)
    s["v"] = s["v"].clone()
    s["v"][2, 1, 77] = bad
    call(s)
    slot = int(s["slots"][2])
    got = ops64.cache_values(s["vc"].cpu(), s["vs"].cpu())[slot // 16, slot % 16]
    assert not np.isfinite(got[1]).all()
    if kv == "int8" or bad == float("inf"):
        assert np.isnan(got[1]).all()
    assert np.isfinite(got[0]).all()


def test_without_norm_or_rotation_it_is_store_kv():
    s = make(40, 8, 2, 64, 16, rot=0, seed=8)
    t = snapshot(s)
    out = call(s, q_weight=False, k_weight=False)
    pa.store_kv(t["k"], t["v"], t["slots"], t["kc"], t["vc"])
    assert torch.equal(out, s["q"])
    assert torch.equal(s["kc"].view(torch.int16), t["kc"].view(torch.int16))
    assert torch.equal(s["vc"].view(torch.int16), t["vc"].view(torch.int16))


def test_q_in_place_and_copied_layouts():
    s = make(33, 8, 2, 128, 16, seed=9, fused=False)
    want = call(s).clone()
    q0 = s["q"].clone()
    s["q"] = q0.clone()
    assert call(s, q_out=s["q"]) is s["q"]
    assert torch.equal(s["q"], want)
    # head-major storage: no token stride describes it, the binding copies
    s["q"] = q0.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(call(s), want)
    # a base that is not 16-byte aligned
    buf = torch.empty(q0.numel() + 1, dtype=torch.bfloat16, device="cuda")
    s["q"] = buf[1:].view(q0.shape)
    s["q"].copy_(q0)
    assert torch.equal(call(s), want)


def test_padding_rows_are_left_as_they_were():
    s = make(8, 4, 2, 128, 16, seed=10)
    s["slots"][6:] = -1
    s["pos"][6:] = -5  # not read
    before = snapshot(s)
    out = torch.full((8, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    call(s, q_out=out)
    assert pa.get_device_error() == 0
    assert (out[6:] == 7.0).all()
    s["pos"][6:] = 0
    check(s, before, out)


def test_positions_and_slots_out_of_range_are_skipped_and_flagged():
    s = make(8, 4, 2, 128, 16, seed=11)
    nslots = s["kc"].shape[0] * 16
    s["pos"][1], s["pos"][2] = 512, -1
    s["slots"][3] = nslots
    before = snapshot(s)
    out = torch.full((8, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    call(s, q_out=out)
    assert pa.get_device_error() == pa.PA_DEVERR_POSITION_RANGE | pa.PA_DEVERR_SLOT_RANGE
    assert (out[1:3] == 7.0).all()  # skipped whole
    q3 = out[3].clone()
    s["slots"][1:4] = -1
    s["pos"][1:3] = 0
    check(s, before, out)
    want, mag = ops64.norm_rope(s["q"][3:4].float().cpu().double().numpy(),
                                s["qw"].float().cpu().double().numpy(), EPS, s["cs"].cpu().numpy(),
                                s["pos"][3:4].cpu().numpy(), False)
    check_rows(q3[None].float().cpu().double().numpy(), want, mag, "q of a token beyond the pool")


def test_other_stream_and_graph_replay():
    s = make(24, 8, 2, 128, 16, seed=12)
    before = snapshot(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros((24, 8, 128), dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(side):
        call(s, q_out=out)
    check(s, before, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.norm_rope_store(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["kc"], s["vc"],
                           q_weight=s["qw"], k_weight=s["kw"], eps=EPS, cos_sin=s["cs"],
                           q_out=out, scores=s["scores"])
    for step in range(3):  # new tokens, positions and slots in place between replays
        s["q"].copy_(torch.randn_like(s["q"]))
        s["k"].copy_(torch.randn_like(s["k"]))
        s["pos"].random_(0, 512)
        s["slots"].copy_(torch.randperm(s["kc"].shape[0] * 16, device="cuda")[:24])
        before = snapshot(s)
        graph.replay()
        torch.cuda.synchronize()
        check(s, before, out)


@pytest.mark.parametrize("kv", ["fp8", "int8"])
@pytest.mark.parametrize("case", [(450, 8, 8, False), (900, 8, 8, True), (520, 24, 20, False),
                                  (1201, 64, 8, False)], ids=lambda c: f"T{c[0]}H{c[1]}kv{c[2]}")
def test_large_8_bit_stores(case, kv):
    # past the first launch bound a warp takes two rounds of two rows, two or four times over:
    # with eight kv heads and more the quantised rows go round that loop as well
    T, H, Hkv, inter = case
    s = make(T, H, Hkv, 128, 16, kv, 128, seed=T)
    s["slots"][T // 3] = -1
    before = snapshot(s)
    out = call(s, inter)
    assert pa.get_device_error() == 0
    check(s, before, out, inter)


@pytest.mark.parametrize("kv", ["fp8", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_every_element_of_a_row_with_a_nan_or_infinity_reads_back_as_nan(kv, bad):
    s = make(6, 2, 2, 128, 16, kv, seed=13)
    s["v"], s["k"] = s["v"].clone(), s["k"].clone()
    s["v"][2, 1, 77] = bad
    s["k"][4, 0, 3] = bad
    call(s)
    for name, t, h in (("v", 2, 1), ("k", 4, 0)):
        slot = int(s["slots"][t])
        got = ops64.cache_values(s[name + "c"].cpu(), s[name + "s"].cpu())[slot // 16, slot % 16]
        assert np.isnan(got[h]).all()
        assert np.isfinite(got[1 - h]).all()
