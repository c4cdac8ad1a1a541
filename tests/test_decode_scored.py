"""pa_decode_scored: out as pa_decode, scores against a plain 64-bit implementation.

Bound on a score. A query-key score s = scale * sum of 128 products of exact
bf16 (or code) values in fp32 differs from the exact one by at most
128 * 2^-23 * sum |q_i k_i| * scale (each addition of the tensor core may
truncate), its scaling by 3 * 2^-24 |s| more; both lie within e = 2^-16 * m,
m = max over the keys of sum |q_i k_i| * scale. A weight
exp(s - max) / sum is then off by at most 2 e relative, plus 2^-21 for the
two exponentials, and the sum over L keys and its merges by (L / 8 + 32) * 2^-24
(a lane adds its own eighth of a block at a time). The additions over the heads
and to the score round 2^-24 of the result each.
"""
import numpy as np
import pytest
import torch

import ops64
import paged_kv_cache_186_gb300 as pa
import workloads as W
from gpu_util import assert_attention_close, to_device

pytestmark = pytest.mark.gpu


def inputs(batch, H, Hkv, D, bs, lens, kv="bf16", seed=0):
    h = W.make_decode(batch, H, Hkv, D, bs, lens, seed=seed, kv_dtype=kv)
    g = to_device(h)
    pa.store_kv(g.k_new, g.v_new, g.slot_mapping, g.k_cache, g.v_cache, g.k_scale_new,
                g.v_scale_new, g.k_scale, g.v_scale)
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(seed)
    nb = g.k_cache.shape[0]
    scores = torch.rand((nb, Hkv, bs), generator=gen).cuda()
    return g, scores


def step(g, scores, **kw):
    out = pa.decode_scored(g.q, g.k_cache, g.v_cache, g.block_tables, g.context_lens, scores,
                           g.scale, k_scale=g.k_scale, v_scale=g.v_scale, **kw)
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    return out


def check(g, before, scores, out, lens, reps=1):
    n64 = lambda t: t.float().cpu().double().numpy()
    kc, vc = (ops64.cache_values(c.cpu(), None if s is None else s.cpu())
              for c, s in ((g.k_cache, g.k_scale), (g.v_cache, g.v_scale)))
    bs = g.k_cache.shape[1]
    want, add, mag = ops64.decode_scored(n64(g.q), kc, vc, g.block_tables.cpu().numpy(), lens,
                                         g.scale, tuple(scores.shape))
    assert_attention_close(out, want, "out")
    add, mag = add * reps, mag * reps
    exact = before.cpu().double().numpy() + add
    got = scores.cpu().double().numpy()
    L = max(max(lens), 1)
    G = g.q.shape[1] // g.k_cache.shape[2]
    tol = (mag * 2.0 ** -15 + add * (2.0 ** -21 + (L / 8 + 32 + G) * 2.0 ** -24)
           + np.abs(exact) * 2.0 ** -24 * reps)
    err = np.abs(got - exact)
    assert (err <= tol).all(), f"scores: {float((err - tol).max()):.3e} past the bound"
    # slots that no sequence sees are untouched
    seen = add > 0
    unseen = torch.from_numpy(~seen)
    tail = np.zeros(scores.shape[::2], bool)
    for b, n in enumerate(lens):
        j = np.arange(n)
        tail[g.block_tables.cpu().numpy()[b][j // bs], j % bs] = True
    untouched = torch.from_numpy(~np.repeat(tail[:, None, :], scores.shape[1], axis=1)) & unseen
    assert torch.equal(scores.cpu()[untouched], before.cpu()[untouched])


CASES = [
    # batch, H, Hkv, D, bs, lens, kv
    (1, 1, 1, 64, 16, [1], "bf16"),
    (4, 8, 2, 64, 16, [1, 17, 33, 100], "bf16"),
    (5, 8, 8, 64, 32, [0, 31, 32, 33, 300], "bf16"),
    (3, 32, 8, 128, 16, [0, 513, 77], "bf16"),
    (3, 24, 8, 128, 32, [1000, 0, 4], "bf16"),         # group 3
    (2, 40, 8, 128, 16, [250, 999], "bf16"),           # group 5
    (2, 14, 2, 128, 16, [250, 60], "bf16"),            # group 7
    (6, 64, 8, 128, 32, [1, 2, 40, 700, 63, 64], "fp8"),
    (4, 16, 4, 128, 16, [15, 16, 17, 500], "fp8"),
    (4, 32, 8, 128, 16, [3, 90, 1025, 0], "int8"),
    (2, 8, 8, 128, 32, [333, 1], "int8"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c[0]}H{c[1]}kv{c[2]}D{c[3]}bs{c[4]}{c[6]}")
def test_matches_decode_and_64_bits(case):
    batch, H, Hkv, D, bs, lens, kv = case
    g, scores = inputs(batch, H, Hkv, D, bs, lens, kv, seed=200 + H + D + bs)
    before = scores.clone()
    out = step(g, scores)
    ref = pa.decode(g.q, g.k_cache, g.v_cache, g.block_tables, g.context_lens, g.scale,
                    k_scale=g.k_scale, v_scale=g.v_scale)
    assert torch.equal(out, ref)
    check(g, before, scores, out, lens)


def test_split_sequences_and_many_short_ones():
    for lens, seed in (([20000, 3, 0, 5000], 230), ([1 + 7 * i % 50 for i in range(300)], 231)):
        g, scores = inputs(len(lens), 8, 2, 128, 16, lens, seed=seed)
        before = scores.clone()
        out = step(g, scores, max_context_len=max(lens))
        check(g, before, scores, out, lens)


def test_slots_behind_the_sequence_may_hold_anything():
    lens = [5, 40, 16]
    g, scores = inputs(3, 8, 2, 128, 16, lens, seed=232)
    bt = g.block_tables.cpu()
    for b, n in enumerate(lens):
        for p in range(n, -(-n // 16) * 16):
            g.k_cache[bt[b, p // 16], p % 16] = float("nan")
            g.v_cache[bt[b, p // 16], p % 16] = float("inf")
            scores[bt[b, p // 16], :, p % 16] = float("nan")
    out = step(g, scores)
    assert torch.isfinite(out.float()).all()
    for b, n in enumerate(lens):
        for p in range(n):
            assert torch.isfinite(scores[bt[b, p // 16], :, p % 16]).all()
        for p in range(n, -(-n // 16) * 16):
            assert torch.isnan(scores[bt[b, p // 16], :, p % 16]).all()


def test_the_weights_of_a_step_sum_to_the_group():
    lens = [700, 64, 1]
    g, scores = inputs(3, 12, 4, 128, 32, lens, seed=233)
    scores.zero_()
    step(g, scores)
    bt = g.block_tables.cpu()
    for b, n in enumerate(lens):
        p = torch.arange(n)
        total = scores.cpu()[bt[b, p // 32].long(), :, p % 32].double().sum(0)
        # 3 heads whose weights each sum to 1 within the bounds above
        assert (total - 3).abs().max().item() <= 3 * (2.0 ** -21 + 2 * (n / 8 + 32) * 2.0 ** -24)


def test_sequences_that_share_blocks_add_up():
    # two sequences over the same prefix blocks, each with a last block of its own
    g, scores = inputs(2, 8, 2, 128, 16, [70, 75], seed=234)
    g.block_tables[1, :4] = g.block_tables[0, :4]
    before = scores.clone()
    out = step(g, scores)
    n64 = lambda t: t.float().cpu().double().numpy()
    _, add, mag = ops64.decode_scored(n64(g.q), n64(g.k_cache), n64(g.v_cache),
                                      g.block_tables.cpu().numpy(), [70, 75], g.scale,
                                      tuple(scores.shape))
    exact = n64(before) + add
    tol = mag * 2.0 ** -15 + add * (2.0 ** -20) + exact * 2.0 ** -23
    assert (np.abs(n64(scores) - exact) <= tol).all()
    assert out.shape == g.q.shape


def test_graph_replays_accumulate_and_two_graphs_share_a_workspace():
    lens = [100, 1000, 37]
    g, scores = inputs(3, 8, 2, 128, 16, lens, seed=235)
    need = pa.decode_scored_workspace_size(g.k_cache, 3, 8, g.block_tables.shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(g.q) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    step(g, scores.clone(), workspace=ws)
    for k in range(2):
        with torch.cuda.graph(graphs[k]):
            pa.decode_scored(g.q, g.k_cache, g.v_cache, g.block_tables, g.context_lens, scores,
                             g.scale, out=outs[k], workspace=ws)
    before = scores.clone()
    for _ in range(3):  # one after the other on one stream
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    check(g, before, scores, outs[0], lens, reps=6)


@pytest.mark.parametrize("H, bs", [(8, 16), (6, 16), (2, 16), (2, 32), (16, 32)])
def test_any_workspace_alignment_and_what_lies_around_it(H, bs):
    lens = [300, 1, 77]
    g, scores = inputs(3, H, 2, 128, bs, lens, seed=240 + H)
    need = pa.decode_scored_workspace_size(g.k_cache, 3, H, g.block_tables.shape[1])
    want = scores.clone()
    step(g, want)
    for shift in (0, 16, 64, 112):
        big = torch.arange(need + 512, device="cuda").to(torch.uint8)
        got = scores.clone()
        step(g, got, workspace=big[128 + shift:128 + shift + need])
        assert torch.equal(got, want)
        ref = torch.arange(need + 512, device="cuda").to(torch.uint8)
        assert torch.equal(big[:128 + shift], ref[:128 + shift])
        assert torch.equal(big[128 + shift + need:], ref[128 + shift + need:])


def test_other_stream_and_repeatability():
    lens = [900, 31, 5, 2048]
    g, scores = inputs(4, 32, 8, 128, 16, lens, seed=236)
    a, b = scores.clone(), scores.clone()
    step(g, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pa.decode_scored(g.q, g.k_cache, g.v_cache, g.block_tables, g.context_lens, b, g.scale)
    side.synchronize()
    # one addition per slot; a segment's parts merge in the order of the parts
    assert torch.equal(a, b)


def test_workspace_and_batch_refusals():
    g, scores = inputs(2, 8, 2, 128, 16, [20, 30], seed=237)
    need = pa.decode_scored_workspace_size(g.k_cache, 2, 8, g.block_tables.shape[1])
    assert need > pa.decode_workspace_size(g.k_cache, 2, 8, g.block_tables.shape[1])
    small = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(pa.PAError, match="WORKSPACE"):
        step(g, scores, workspace=small)
    B = 16385
    q = torch.zeros((B, 1, 64), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((4, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    assert pa.decode_scored_workspace_size(kc, B, 1, 1) == 0
    with pytest.raises(pa.PAError, match="UNSUPPORTED"):
        pa.decode_scored(q, kc, kc.clone(), bt, bt[:, 0].contiguous(),
                         torch.zeros((4, 1, 16), device="cuda"), 0.1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_key_that_is_not_finite_spoils_its_own_score_only(bad):
    # in a sequence that one warp holds and in one that is split over many
    lens = [40, 5000, 700]
    g, scores = inputs(3, 8, 2, 128, 16, lens, seed=240)
    bt = g.block_tables.cpu().long()
    before = scores.clone()
    g.q.abs_()  # a key of +infinity in one dim scores +infinity, not NaN
    clean = scores.clone()
    ref = step(g, clean)
    for b, p in ((0, 21), (1, 3333)):
        g.k_cache[bt[b, p // 16], p % 16, 1, 5] = bad
    out = step(g, scores)
    assert torch.isnan(out[:2, 4:].float()).all()
    assert torch.equal(out[:2, :4], ref[:2, :4]) and torch.equal(out[2], ref[2])
    want = clean.clone()
    for b, p in ((0, 21), (1, 3333)):
        blocks = bt[b, :-(-lens[b] // 16)].cuda()
        want[blocks, 1] = before[blocks, 1]
        want[bt[b, p // 16], 1, p % 16] = float("nan")
    assert torch.equal(torch.isnan(scores), torch.isnan(want))
    assert torch.equal(scores.nan_to_num(-1.0), want.nan_to_num(-1.0))
