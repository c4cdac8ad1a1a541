"""pa_decode_shared against a plain 64-bit implementation (the library's attention tolerance)
and against pa_decode of the same batch."""
import numpy as np
import pytest
import torch

import paged_kv_cache_186_gb300 as pa
from gpu_util import assert_attention_close
from shared_util import decode64, make, n64
from test_prefill_shared import weights_of_few_keys_hold

pytestmark = pytest.mark.gpu


def run(s, **kw):
    out = pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.cu_groups,
                           s.prefix_lens, s.scale, always=True, k_scale=s.k_scale, v_scale=s.v_scale, **kw)
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    return out


def plain(s):
    return pa.decode(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.scale, k_scale=s.k_scale,
                     v_scale=s.v_scale)


CASES = [
    # groups [(prefix, lengths)], H, Hkv, D, bs, kv
    ([(64, [65, 70, 100])], 8, 2, 128, 16, "bf16"),
    ([(1, [1])], 1, 1, 128, 16, "bf16"),
    ([(16, [16, 17, 33])], 4, 4, 64, 16, "bf16"),
    ([(500, [501, 700, 0, 512, 530])], 8, 2, 128, 32, "bf16"),   # a padding row
    ([(128, [129] * 40)], 8, 1, 128, 16, "bf16"),                # 320 rows: three tiles
    ([(257, [300] * 33), (1000, [1001, 1024]), (48, [49] * 7)], 12, 4, 128, 16, "bf16"),  # group 3
    ([(130, [131] * 20)], 10, 2, 128, 16, "bf16"),               # group 5
    ([(300, [301 + i for i in range(19)])], 14, 2, 64, 32, "bf16"),  # group 7, head_dim 64
    ([(1000, [1100] * 70)], 8, 2, 64, 16, "bf16"),
    ([(640, [641, 1300, 650, 0])], 16, 2, 128, 32, "fp8"),
    ([(100, [101] * 36), (333, [400, 334])], 8, 1, 128, 16, "fp8"),
    ([(640, [641, 1300, 650])], 6, 2, 128, 16, "int8"),
    ([(96, [97] * 50)], 8, 1, 128, 32, "int8"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}g{sum(len(x[1]) for x in c[0])}"
                         f"H{c[1]}kv{c[2]}D{c[3]}bs{c[4]}{c[5]}")
def test_matches_64_bits_and_decode(case):
    groups, H, Hkv, D, bs, kv = case
    s = make(groups, H, Hkv, D, bs, kv, seed=500 + H + D + bs + len(groups))
    out = run(s)
    want = decode64(s)
    assert_attention_close(out, want, str(case))
    assert_attention_close(plain(s), want, "decode")
    for b, n in enumerate(s.lens):
        if n == 0:
            assert (out[b] == 0).all()


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 384, 1 << 20])
@pytest.mark.parametrize("bs", [16, 32])
def test_prefix_lengths_around_blocks_and_tiles(prefix, bs):
    s = make([(prefix, [300, 290, 299])], 8, 2, 128, bs, seed=520 + prefix % 97)
    assert_attention_close(run(s), decode64(s), f"prefix {prefix}")


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_sequences_shorter_than_the_prefix_and_padding(kv):
    # the first rows of the group are padding and too short to name the blocks; a group of short
    # sequences only shares nothing; rows of padding hold anything in the table
    s = make([(200, [0, 30, 3, 205, 0, 200, 144]), (500, [40, 0, 20]), (64, [0, 0])], 8, 2, 128, 16,
             kv, seed=540)
    s.bt[s.context_lens == 0] = 1 << 30
    out = run(s)
    assert_attention_close(out, decode64(s), "short")
    assert (out[s.context_lens == 0] == 0).all()


def test_groups_that_are_empty_missing_or_leave_sequences_out():
    s = make([(64, [80, 81]), (32, []), (100, [120])], 8, 2, 64, 16, seed=541,
             outside=((50, 0, 7), (300, 12)))
    want = decode64(s)
    assert_attention_close(run(s), want, "outside")
    s.cu_groups, s.prefix_lens = s.cu_groups[:1], s.prefix_lens[:0]
    assert_attention_close(run(s), want, "no groups")


def test_group_bounds_that_do_not_ascend_or_lie_outside():
    s = make([(64, [80, 81, 90, 70])], 8, 2, 128, 16, seed=542)
    want = decode64(s)
    for cu in ([-7, 3, 1, 900], [0, 4, 2, 4], [3, 3, 3, 3], [9, 9, 9, 9], [0, 1 << 30, -5, 4]):
        s.cu_groups = torch.tensor(cu, dtype=torch.int32).cuda()
        s.prefix_lens = torch.tensor([64, 64, 64], dtype=torch.int32).cuda()
        assert_attention_close(run(s), want, str(cu))
    s.cu_groups = torch.tensor([0, 4], dtype=torch.int32).cuda()
    for p in (-1, -(1 << 31), (1 << 31) - 1):
        s.prefix_lens = torch.tensor([p], dtype=torch.int32).cuda()  # (too long: nothing shared)
        assert_attention_close(run(s), want, f"prefix {p}")


def test_slots_behind_a_sequence_may_hold_anything():
    s = make([(70, [75, 100, 81]), (40, [41, 64])], 8, 2, 128, 16, seed=543)
    bt = s.bt.cpu()
    for b, n in enumerate(s.lens):
        for p in range(n, -(-n // 16) * 16):
            s.k_cache[bt[b, p // 16], p % 16] = float("nan")
            s.v_cache[bt[b, p // 16], p % 16] = float("inf")
    assert_attention_close(run(s), decode64(s), "tails")


@pytest.mark.parametrize("kv, D", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("int8", 128)])
def test_long_prefix_many_sequences(kv, D):
    s = make([(20011, [20011 + 37 * i for i in range(1, 18)]), (700, [701 + i for i in range(30)])],
             8, 2, D, 16, kv, seed=544, spread=2.0)
    assert_attention_close(run(s), decode64(s), "long")


@pytest.mark.parametrize("rows", [3, 60])
def test_weight_on_few_keys(rows):
    # a few keys of the prefix and of the sequences' own draw nearly all of the weight
    s = make([(2000, [2001 + 5 * i for i in range(rows)])], 8, 1, 128, 16, seed=545, spread=2.0)
    bt = s.bt.cpu()
    for p in (0, 1, 130, 1999):
        s.k_cache[bt[0, p // 16].item(), p % 16] *= 4
    assert_attention_close(run(s), decode64(s), "few keys")


def test_scores_far_apart_between_prefix_and_own_keys():
    # whole parts of the softmax vanish against others, in either order
    for big in (0, 1):
        s = make([(256, [300, 280, 270])], 8, 2, 128, 16, seed=546 + big)
        blocks = s.bt[:, :16] if big == 0 else s.bt[:, 16:]
        blocks = blocks[blocks >= 0].long()
        s.k_cache[blocks.unique()] *= 60
        assert_attention_close(run(s), decode64(s), f"far {big}")


def test_equal_keys_give_the_mean():
    s = make([(512, [600] * 9)], 8, 2, 128, 16, seed=548)
    s.k_cache[:] = s.k_cache[0, 0, 0]
    assert_attention_close(run(s), decode64(s), "mean")


def test_length_bound_cuts_sequences():
    s = make([(200, [300, 250, 210])], 8, 2, 128, 16, seed=549)
    out = run(s, max_context_len=230)
    s.lens = [min(n, 230) for n in s.lens]
    assert_attention_close(out, decode64(s), "bound")
    out = run(s, max_context_len=100)  # below the prefix
    s.lens = [100] * 3
    assert_attention_close(out, decode64(s), "bound below the prefix")


def test_repeats_other_streams_outputs_and_strided_inputs():
    s = make([(1500, [1501 + 31 * i for i in range(25)]), (80, [81, 300])], 32, 8, 128, 16, seed=550)
    a = run(s)
    need = pa.decode_shared_workspace_size(s.k_cache, 27, 32, s.bt.shape[1], 2)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    assert run(s, out=b, workspace=ws) is b
    assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.cu_groups,
                             s.prefix_lens, s.scale, always=True)
    side.synchronize()
    assert torch.equal(a, c)
    wide = torch.cat([s.bt, s.bt], dim=1)[:, :s.bt.shape[1]]
    q = s.q.transpose(0, 1).contiguous().transpose(0, 1)
    lens = torch.stack([s.context_lens] * 2, dim=1)[:, 0]
    d = pa.decode_shared(q, s.k_cache, s.v_cache, wide, lens, s.cu_groups, s.prefix_lens, s.scale, always=True)
    assert torch.equal(a, d)


@pytest.mark.parametrize("shift", [0, 16, 112])
def test_the_workspace_and_what_lies_around_it(shift):
    s = make([(300, [301, 310, 350]), (90, [91] * 40)], 8, 2, 128, 16, seed=551)
    need = pa.decode_shared_workspace_size(s.k_cache, 43, 8, s.bt.shape[1], 2)
    want = run(s)
    ref = torch.arange(need + 512, device="cuda").to(torch.uint8)
    big = ref.clone()
    out = run(s, workspace=big[128 + shift:128 + shift + need])
    assert torch.equal(out, want)
    assert torch.equal(big[:128 + shift], ref[:128 + shift])
    assert torch.equal(big[128 + shift + need:], ref[128 + shift + need:])
    with pytest.raises(pa.PAError, match="WORKSPACE"):
        run(s, workspace=big[128 + shift:128 + shift + need - 1])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_graph_replays_with_lengths_and_groups_rewritten(kv):
    s = make([(320, [330, 340, 350, 360]), (64, [100, 90, 70])], 8, 2, 128, 16, kv, seed=552)
    need = pa.decode_shared_workspace_size(s.k_cache, 7, 8, s.bt.shape[1], 2, k_scale=s.k_scale,
                                           v_scale=s.v_scale)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(s.q) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    run(s, workspace=ws)
    for k in range(2):  # two graphs that share the workspace
        with torch.cuda.graph(graphs[k]):
            pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.cu_groups,
                             s.prefix_lens, s.scale, always=True, out=outs[k], workspace=ws, k_scale=s.k_scale,
                             v_scale=s.v_scale)
    gen = torch.Generator().manual_seed(1)
    for step in range(4):
        s.q.copy_(torch.randn(s.q.shape, generator=gen))
        if step == 1:
            s.context_lens.copy_(torch.tensor([321, 340, 0, 322, 70, 65, 0], dtype=torch.int32))
        if step == 2:
            s.prefix_lens.copy_(torch.tensor([160, 0], dtype=torch.int32))
        if step == 3:
            s.cu_groups.copy_(torch.tensor([1, 4, 4], dtype=torch.int32))
        s.lens = s.context_lens.tolist()
        for o, graph in zip(outs, graphs):
            o.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        assert pa.get_device_error() == 0
        want = decode64(s)
        assert_attention_close(outs[0], want, f"step {step}")
        assert torch.equal(outs[0], outs[1])
        assert torch.equal(outs[0], run(s))


def test_bad_block_ids_are_flagged_and_spoil_their_group_only():
    s = make([(320, [330, 340]), (64, [100, 90, 70])], 8, 2, 128, 16, seed=553)
    want = decode64(s)
    for bad in (-1, 1 << 30):
        s.bt[0, 3] = bad
        out = pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.cu_groups,
                               s.prefix_lens, s.scale, always=True)
        assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_RANGE
        assert_attention_close(out[2:], want[2:], "other group")


def test_large_batches_of_few_heads_and_many_groups():
    # 600 sequences in 150 groups of four
    groups = [(48 + 16 * (i % 5), [50 + 16 * (i % 5) + j for j in range(4)]) for i in range(150)]
    s = make(groups, 2, 1, 64, 16, seed=554)
    assert_attention_close(run(s), decode64(s), "many groups")


def test_batches_and_groups_above_the_limit_are_refused():
    B = 16385
    kc = torch.zeros((4, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((B, 1, 64), dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, B], dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    assert pa.decode_shared_workspace_size(kc, B, 1, 1, 1) == 0
    with pytest.raises(pa.PAError, match="UNSUPPORTED"):
        pa.decode_shared(q, kc, kc.clone(), bt, bt[:, 0].contiguous(), cu, one, 0.1)
    assert pa.decode_shared_workspace_size(kc, 4, 1, 1, B) == 0
    many = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(pa.PAError, match="UNSUPPORTED"):
        pa.decode_shared(q[:4], kc, kc.clone(), bt[:4], bt[:4, 0].contiguous(), many, many[1:], 0.1)


def test_an_empty_batch():
    s = make([(16, [20])], 8, 2, 128, 16, seed=555)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pa.decode_shared(s.q[:0], s.k_cache, s.v_cache, s.bt[:0], s.context_lens[:0], cu,
                           cu[:0], s.scale)
    assert out.shape == (0, 8, 128)


def test_seeded_random_batches():
    r = np.random.default_rng(7)
    for i in range(24):
        kv, D = [("bf16", 128), ("bf16", 64), ("fp8", 128), ("int8", 128)][i % 4]
        bs, Hkv, G = int(r.choice([16, 32])), int(r.choice([1, 2, 4])), int(r.integers(1, 9))
        groups = []
        for _ in range(int(r.integers(1, 5))):
            p = int(r.integers(0, 900))
            groups.append((p, [int(n) for n in p + r.integers(-p // 2, 300, int(r.integers(1, 40)))]))
        groups = [(p, [max(n, 0) for n in ls]) for p, ls in groups]
        s = make(groups, G * Hkv, Hkv, D, bs, kv, seed=600 + i, outside=((5,), ()) if i % 3 else ((), ()))
        bound = max(s.lens) if i % 2 else 0
        assert_attention_close(run(s, max_context_len=bound), decode64(s), f"case {i}: {groups}")


@pytest.mark.parametrize("kv, D, bs", [("bf16", 64, 16), ("bf16", 64, 32), ("bf16", 128, 16),
                                       ("fp8", 128, 32), ("int8", 128, 16)])
@pytest.mark.parametrize("seqs", [1, 3, 40])
def test_many_groups_of_a_few_key_tiles_over_and_over(kv, D, bs, seqs):
    # segments of one to twenty key tiles: every CTA walks many pieces, and the stages of its rings
    # are handed from one half to the other in every order; repeated, since a wait that could
    # be passed early or never would depend on timing
    r = np.random.default_rng(D + bs + seqs)
    groups = []
    for _ in range(24):
        p = int(r.integers(1, 2600))
        groups.append((p, [p + int(r.integers(1, 60)) for _ in range(seqs)]))
    s = make(groups, 8, 4, D, bs, kv, seed=560 + seqs)
    first = run(s)
    assert_attention_close(first, plain(s).double().cpu().numpy(), "against decode")
    for _ in range(60):
        out = pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.cu_groups,
                               s.prefix_lens, s.scale, always=True, k_scale=s.k_scale, v_scale=s.v_scale)
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    assert torch.equal(out, first)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_values_of_any_magnitude(kv):
    # V (or its scales) from 2^-30 to 2^40 between tiles and heads: the factor that brings V into
    # f16 moves with them; zeros leave it where it is
    s = make([(1200, [1201, 1300, 1250])], 8, 2, 128, 16, kv, seed=570)
    blocks = s.bt[0, :75].long()
    t = s.v_cache if kv == "bf16" else s.v_scale
    ref = t.clone()
    for shifts in ([0, -30, 40, 5], [40, 0, -30, 12], [-30, -30, -30, -30], [100, -20, -90, 3],
                   [-90, 3, 100, -20], [-75, -60, -75, -75]):
        t.copy_(ref)
        for i, e in enumerate(shifts):
            part = blocks[i * 19:(i + 1) * 19]
            t[part] = t[part] * 2.0 ** e
        t[blocks[20:30]] = 0
        want = decode64(s)
        got = n64(run(s))
        # relative to the largest value a row could have from the keys it weighs
        top = np.abs(want).max(axis=-1, keepdims=True)
        assert (np.abs(got - want) <= top * 2.0 ** -6).all()
        assert np.linalg.norm(got - want) <= 5e-3 * np.linalg.norm(want)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_value_that_is_not_finite_spoils_its_dim_only(bad):
    s = make([(300, [310, 305])], 8, 2, 128, 16, seed=571)
    want = decode64(s)
    s.v_cache[s.bt[0, 5].item(), 3, 1, 7] = bad
    out = run(s).float()
    assert not torch.isfinite(out[:, 4:, 7]).any()
    out[:, 4:, 7] = torch.from_numpy(want[:, 4:, 7])
    assert_attention_close(out, want, "the other dims")


def test_blocks_beyond_2_to_the_32_elements():
    # the same shared and own blocks at the front of a small pool and at the end of a large one
    s = make([(200, [210, 230, 201]), (64, [70])], 8, 8, 128, 32, seed=572)
    small = run(s)
    per = 32 * 8 * 128
    nb = (1 << 32) // per + 64
    need = s.k_cache.shape[0]
    big_k, big_v = (torch.empty((nb, 32, 8, 128), dtype=torch.bfloat16, device="cuda")
                    for _ in range(2))
    big_k[nb - need:], big_v[nb - need:] = s.k_cache, s.v_cache
    bt = torch.where(s.bt >= 0, s.bt + (nb - need), s.bt)
    out = pa.decode_shared(s.q, big_k, big_v, bt, s.context_lens, s.cu_groups, s.prefix_lens, s.scale, always=True)
    torch.cuda.synchronize()
    assert torch.equal(out, small)


@pytest.mark.parametrize("kv, batch, prefix, shares", [("bf16", 4, 1000, False), ("bf16", 40, 8000, True),
                                                       ("int8", 2, 400, False), ("int8", 20, 2000, True)])
def test_without_always_small_calls_are_decode(kv, batch, prefix, shares):
    s = make([(prefix, [prefix + 5 + i for i in range(batch)])], 32, 8, 128, 16, kv, seed=580)
    out = pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.cu_groups,
                           s.prefix_lens, s.scale, k_scale=s.k_scale, v_scale=s.v_scale)
    always, ref = run(s), plain(s)
    torch.cuda.synchronize()
    assert torch.equal(out, always if shares else ref)
    assert not torch.equal(always, ref)
    assert_attention_close(out, ref.double().cpu().numpy(), "decode")


@pytest.mark.parametrize("kv, D", [("bf16", 128), ("bf16", 64), ("fp8", 128)])
def test_long_own_contexts(kv, D):
    # own segments of more parts than the merge takes (merged before it), next to short ones
    s = make([(64, [21000, 70, 5003, 64]), (33, [30, 9000])], 8, 2, D, 16, kv, seed=590,
             outside=((15000,), (3,)))
    for bound in (0, 21000):
        assert_attention_close(run(s, max_context_len=bound), decode64(s), "long own")


def test_two_calls_at_once_on_two_streams():
    cases = [make([(3000, [3010 + i for i in range(40)])], 8, 2, 128, 16, seed=591),
             make([(700, [720, 705, 800]), (64, [65] * 9)], 16, 2, 128, 32, "fp8", seed=592)]
    want = [run(s) for s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(25):
        for s, stream, out in zip(cases, streams, outs):
            with torch.cuda.stream(stream):
                out.append(pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens,
                                            s.cu_groups, s.prefix_lens, s.scale, always=True,
                                            k_scale=s.k_scale, v_scale=s.v_scale))
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    for w, out in zip(want, outs):
        assert all(torch.equal(w, o) for o in out)


def test_a_workspace_for_the_most_sequences_and_groups_serves_fewer():
    # fewer groups may have two row tiles a segment, whose partials are twice as large; larger
    # batches fewer partial slots
    kc = torch.zeros((4, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    small = torch.zeros((4, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    for cache, H, batches in ((kc, 32, [1, 7, 31, 32, 33, 64, 65, 200, 256, 257, 960]),
                              (small, 1, [1, 128, 129, 300, 5000, 9999, 16384]),
                              (small, 3, [42, 43, 84, 86])):
        groups = [0, 1, 2, 3, 8, 30, 31, 64, 1000, 16384]
        for bound in (0, 40):
            need = torch.tensor([[pa.decode_shared_workspace_size(cache, b, H, 64, g, bound)
                                  for g in groups] for b in batches])
            assert (need > 0).all()
            assert (need.diff(dim=0) >= 0).all() and (need.diff(dim=1) >= 0).all(), need
            if bound:
                assert (need <= wide).all()
            wide = need
    s = make([(200, [201 + i for i in range(64)])], 32, 8, 128, 16, seed=593)
    want = decode64(s)
    ws = torch.full((pa.decode_shared_workspace_size(s.k_cache, 64, 32, s.bt.shape[1], 2),), 255,
                    dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for cu in ([0, 30, 64], [0, 64], [3, 50]):
        s.cu_groups, s.prefix_lens = i32(cu), i32([200] * (len(cu) - 1))
        assert_attention_close(run(s, workspace=ws), want, f"groups {cu}")
    s.q, s.bt, s.context_lens, s.lens = s.q[:9], s.bt[:9], s.context_lens[:9], s.lens[:9]
    s.cu_groups = i32([0, 9])
    s.prefix_lens = s.prefix_lens[:1]
    assert_attention_close(run(s, workspace=ws), want[:9], "9 sequences")


def test_the_workspace_is_no_larger_than_documented():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for D, Hkv, H in ((128, 8, 32), (64, 8, 64), (128, 1, 3), (64, 4, 20), (128, 8, 8)):
        kc = torch.zeros((4, 16, Hkv, D), dtype=torch.bfloat16, device="cuda")
        for rows in (1, 7, 64, 960, 1024, 16384):
            for g in (1, 2, 30, 256, 8192):
                if g > rows:
                    continue
                floats = (D + 2) * (2 * H * rows + 256 * Hkv * g + 256 * sms)
                decode = pa.decode_workspace_size(kc, min(rows, 256), H, 64)
                need = pa.decode_shared_workspace_size(kc, rows, H, 64, g)
                assert need - decode <= 1.1 * 4 * floats, (D, Hkv, H, rows, g)
                if D == 128 and H // Hkv in (1, 2, 4, 8, 16):
                    need = pa.prefill_shared_workspace_size(kc, rows, H, g)
                    assert need <= 1.1 * 4 * floats, (D, Hkv, H, rows, g)


@pytest.mark.parametrize("D, seqs", [(64, 700), (128, 400), (64, 500)])
def test_a_team_of_lanes_for_each_row(D, seqs):
    # above 16 warps of rows an SM the merge gives a row to a team of lanes, below it to a CTA: with 8
    # kv heads on 152 SMs from 608 rows of head_dim 64, 304 of 128
    lens = [[33 + (7 * i + j) % 60 for j in range(seqs // 4)] for i in range(4)]
    lens[2][5] = lens[3][0] = 0
    s = make([(32 + 16 * i, [n + 16 * i if n else 0 for n in ls]) for i, ls in enumerate(lens)], 16, 8,
             D, 16, seed=594)
    out = run(s)
    assert_attention_close(out, decode64(s), "teams")
    assert (out[s.context_lens == 0] == 0).all()


@pytest.mark.parametrize("groups", [512, 513, 1023, 1024, 1025, 2049])
@pytest.mark.parametrize("order", ["ascending", "mixed"])
def test_more_groups_than_fit_the_plan_or_one_of_its_passes(groups, order):
    # one prefix for all sequences, so that any partition of them is one of groups that share it:
    # bounds of empty groups, and such that fall back or lie outside
    r = np.random.default_rng(groups)
    n = 1300
    s = make([(50, [49 + int(x) for x in r.integers(0, 40, n)])], 2, 1, 64, 16, seed=595)
    cu = np.sort(r.integers(0, n + 1, groups + 1))
    if order == "mixed":
        at = r.integers(0, groups + 1, groups // 5)
        cu[at] = r.integers(-50, n, len(at))
        cu[-3:] = n, n + 9, 5
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    s.cu_groups, s.prefix_lens = i32(cu), i32(r.integers(-5, 51, groups))
    assert_attention_close(run(s), decode64(s), f"{groups} groups")


@pytest.mark.parametrize("kv, prefix, own, width", [("bf16", 16, 2000, 0), ("bf16", 30, 100, 2048),
                                                    ("fp8", 40, 700, 0), ("int8", 5, 400, 0)])
def test_without_always_a_short_prefix_of_long_contexts(kv, prefix, own, width):
    # the host's bound takes the whole contexts for shared
    s = make([(prefix, [prefix + own - 3 * i for i in range(33)])], 32, 8, 128, 16, kv, seed=596)
    if width:
        s.bt = torch.cat([s.bt, s.bt.new_full((33, width // 16 - s.bt.shape[1]), -1)], dim=1)
    out = pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.cu_groups,
                           s.prefix_lens, s.scale, k_scale=s.k_scale, v_scale=s.v_scale)
    assert_attention_close(out, decode64(s), "short prefix")


@pytest.mark.parametrize("where", ["own", "shared", "both"])
def test_weights_of_few_dominant_keys_keep_more_bits_than_bf16(where):
    # (bounds: beside the prefill's test; the own keys' weights are two bf16 terms here too)
    weights_of_few_keys_hold(where, [1] * 200, run, decode64)


@pytest.mark.parametrize("group", [3, 5, 6, 7, 4])
@pytest.mark.parametrize("kv, D, seqs", [("bf16", 128, 24), ("bf16", 64, 150), ("fp8", 128, 60),
                                         ("int8", 128, 9)])
def test_repeats_do_not_depend_on_what_shared_memory_holds(group, kv, D, seqs):
    # 128 / group tokens leave rows of a tile's Q unwritten for these groups: calls of four heads in
    # between fill all rows with other magnitudes
    s = make([(2700, [2701 + 3 * i for i in range(seqs)])], group * 2, 2, D, 16, kv, seed=597, spread=2.0)
    t = make([(1500, [1510 + i for i in range(seqs + 40)])], 8, 2, D, 16, kv, seed=598)
    first = run(s)
    assert_attention_close(first, decode64(s), "first")
    q = t.q.clone()
    for f in (0.0, 1.0, 30.0, -7.0, 0.1, 100.0, 3.0, 10.0):
        t.q.copy_(q * f)
        run(t)
        assert torch.equal(run(s), first), f
