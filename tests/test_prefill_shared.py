"""pa_prefill_shared against a plain 64-bit implementation (the library's attention tolerance)
and against pa_prefill_varlen of the same batch."""
import numpy as np
import pytest
import torch

import paged_kv_cache_186_gb300 as pa
from gpu_util import assert_attention_close
from shared_util import make, n64, prefill64

pytestmark = pytest.mark.gpu


def run(s, **kw):
    kw.setdefault("max_q_len", max(s.new, default=0))
    out = pa.prefill_shared(s.q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k, s.cu_groups,
                            s.prefix_lens, s.scale, **{"always": True, **kw})
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    return out


CASES = [
    # groups [(prefix, kv lengths)], new tokens, H, Hkv, bs
    ([(64, [70, 90, 65])], [6, 20, 1], 8, 2, 16),
    ([(1, [1])], [1], 1, 1, 16),
    ([(300, [310, 305, 400])], [10, 5, 100], 32, 8, 32),
    ([(128, [140] * 20)], [3] * 20, 4, 1, 16),
    ([(500, [501 + 3 * i for i in range(9)])], [1 + i for i in range(9)], 16, 2, 16),   # group 8
    ([(333, [400, 350, 334])], [64, 17, 1], 16, 1, 32),                                 # group 16
    ([(200, [300, 290]), (40, [41, 60, 50])], [70, 33, 1, 20, 10], 2, 2, 16),           # group 1
    ([(1000, [1300, 1200])], [300, 129], 8, 4, 16),                                     # group 2
]


@pytest.mark.parametrize("bound", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}g{len(c[1])}H{c[2]}kv{c[3]}bs{c[4]}")
def test_matches_64_bits_and_prefill_varlen(case, bound):
    groups, new, H, Hkv, bs = case
    s = make(groups, H, Hkv, 128, bs, seed=700 + H + bs, new=new)
    want = prefill64(s)
    assert_attention_close(run(s, max_q_len=max(new) if bound else 0), want, str(case))
    ref = pa.prefill_varlen(s.q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k, s.scale)
    assert_attention_close(ref, want, "prefill_varlen")


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 200, 256, 299, 1 << 20])
@pytest.mark.parametrize("new", [[1, 1, 1], [5, 40, 64], [300, 290, 299]])
def test_prefix_lengths_with_new_tokens_inside_and_behind(prefix, new):
    # the last form has no cached keys: most of the new tokens lie within the prefix
    s = make([(prefix, [300, 290, 299])], 8, 2, 128, 16, seed=720 + prefix % 89, new=new)
    assert_attention_close(run(s), prefill64(s), f"prefix {prefix}")


def test_sequences_without_new_tokens_short_ones_and_rows_behind_the_last():
    s = make([(200, [0, 30, 205, 200, 144, 90]), (500, [40, 20]), (32, [])], 8, 2, 128, 16, seed=740,
             new=[0, 3, 5, 1, 0, 9, 40, 2])
    want = prefill64(s)
    T = s.q.shape[0]
    q = torch.cat([s.q, s.q[:7]])  # rows behind the last sequence
    out = torch.full_like(q, 3.0)
    pa.prefill_shared(q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k, s.cu_groups, s.prefix_lens,
                      s.scale, max_q_len=40, out=out, always=True)
    torch.cuda.synchronize()
    assert_attention_close(out[:T], want, "short")
    assert (out[T:] == 3.0).all()


def test_sequences_outside_the_groups():
    s = make([(64, [80, 81]), (100, [120])], 8, 2, 128, 16, seed=741, new=[5, 7, 10, 2, 20, 12],
             outside=((50, 7), (300,)))
    want = prefill64(s)
    assert_attention_close(run(s), want, "outside")
    s.cu_groups, s.prefix_lens = s.cu_groups[:1], s.prefix_lens[:0]
    assert_attention_close(run(s), want, "no groups")


def test_more_new_tokens_than_keys():
    # invalid input, as for prefill_varlen: the cached length is 0, keys are clamped
    s = make([(32, [40, 20, 0])], 8, 2, 128, 16, seed=742, new=[60, 3, 4])
    assert_attention_close(run(s), prefill64(s), "clamped")


@pytest.mark.parametrize("rows", [3, 60])
def test_weight_on_few_keys(rows):
    s = make([(2000, [2001 + 5 * i for i in range(rows)])], 8, 2, 128, 16, seed=745, spread=2.0,
             new=[1 + i % 4 for i in range(rows)])
    bt = s.bt.cpu()
    for p in (0, 1, 100, 1999):
        s.k_cache[bt[0, p // 16].item(), p % 16] *= 4
    assert_attention_close(run(s), prefill64(s), "few keys")


def test_long_prefix_and_long_questions():
    s = make([(9001, [9001 + 200, 9001 + 77, 9400]), (3000, [3300, 3001])], 8, 2, 128, 32, seed=746,
             new=[200, 77, 260, 300, 1], spread=2.0)
    assert_attention_close(run(s), prefill64(s), "long")


def test_repeats_streams_workspaces_and_graphs():
    s = make([(700, [701 + 9 * i for i in range(12)]), (80, [90, 300])], 32, 8, 128, 16, seed=747,
             new=[1 + i % 7 for i in range(12)] + [10, 150])
    a = run(s)
    assert_attention_close(a, prefill64(s), "first")
    T = s.q.shape[0]
    need = pa.prefill_shared_workspace_size(s.k_cache, T, 32, 2)
    ref = torch.arange(need + 512, device="cuda").to(torch.uint8)
    for shift in (0, 16, 112):
        big = ref.clone()
        ws = big[128 + shift:128 + shift + need]
        assert torch.equal(run(s, workspace=ws), a)
        assert torch.equal(big[:128 + shift], ref[:128 + shift])
        assert torch.equal(big[128 + shift + need:], ref[128 + shift + need:])
        with pytest.raises(pa.PAError, match="WORKSPACE"):
            run(s, workspace=ws[:-1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = pa.prefill_shared(s.q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k, s.cu_groups,
                              s.prefix_lens, s.scale, max_q_len=150, always=True)
    side.synchronize()
    assert torch.equal(a, c)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(s.q) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for k in range(2):
        with torch.cuda.graph(graphs[k]):
            pa.prefill_shared(s.q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k, s.cu_groups,
                              s.prefix_lens, s.scale, max_q_len=150, out=outs[k], workspace=ws,
                              always=True)
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a) and torch.equal(outs[1], a)


def test_bad_block_ids_are_flagged_and_spoil_their_group_only():
    s = make([(320, [330, 340]), (64, [100, 90])], 8, 2, 128, 16, seed=748, new=[4, 9, 30, 1])
    want = prefill64(s)
    for bad in (-1, 1 << 30):
        s.bt[0, 3] = bad
        out = pa.prefill_shared(s.q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k, s.cu_groups,
                                s.prefix_lens, s.scale, max_q_len=30, always=True)
        assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_RANGE
        assert_attention_close(out[13:], want[13:], "other group")


def test_a_decode_step_is_a_prefill_of_one_token_each():
    s = make([(500, [501 + 17 * i for i in range(20)])], 8, 2, 128, 16, seed=749, new=[1] * 20)
    dec = pa.decode_shared(s.q, s.k_cache, s.v_cache, s.bt, s.context_lens, s.cu_groups,
                           s.prefix_lens, s.scale, always=True)
    want = prefill64(s)
    assert_attention_close(run(s), want, "prefill")
    assert_attention_close(dec, want, "decode")


def test_seeded_random_batches():
    r = np.random.default_rng(8)
    for i in range(20):
        bs, Hkv, G = int(r.choice([16, 32])), int(r.choice([1, 2, 4])), int(r.choice([1, 2, 4, 8, 16]))
        groups, new = [], []
        for _ in range(int(r.integers(1, 4))):
            p = int(r.integers(0, 700))
            ls = [max(0, int(n)) for n in p + r.integers(-p // 2, 200, int(r.integers(1, 14)))]
            groups.append((p, ls))
            new += [min(n, int(r.integers(0, int(r.choice([3, 30, 150]))))) for n in ls]
        if sum(new) == 0:
            new[0] = 1 if groups[0][1][0] else 0
        if sum(new) == 0:
            continue
        s = make(groups, G * Hkv, Hkv, 128, bs, seed=800 + i, new=new)
        assert_attention_close(run(s, max_q_len=max(new) if i % 2 else 0), prefill64(s),
                               f"case {i}: {groups} {new}")


@pytest.mark.parametrize("new, prefix, shares", [([200, 256, 130], 600, False), ([3] * 40, 6000, True)])
def test_without_always_calls_that_would_not_gain_are_prefill(new, prefix, shares):
    s = make([(prefix, [prefix + n + 9 for n in new])], 32, 8, 128, 16, seed=760, new=new)
    ref = pa.prefill_varlen(s.q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k, s.scale,
                            max_q_len=max(new))
    always, out = run(s), run(s, always=False)
    assert torch.equal(out, always) == shares
    assert_attention_close(out, ref.double().cpu().numpy(), "prefill_varlen")
    if not shares:  # as the windowed prefill computes it, whose window keeps every key
        win = pa.prefill_window(s.q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k, s.scale, 1 << 30,
                                max_q_len=max(new))
        assert torch.equal(out, win)


def test_the_choice_follows_the_lengths_and_mixes_with_sequences_outside():
    # every small case of above again without `always`: the rows are written by one kernel or
    # the other, those without any key by either
    for case in CASES:
        groups, new, H, Hkv, bs = case
        s = make(groups, H, Hkv, 128, bs, seed=770 + H + bs, new=new)
        assert_attention_close(run(s, always=False), prefill64(s), str(case))
    s = make([(64, [80, 81, 0]), (100, [120])], 8, 2, 128, 16, seed=771,
             new=[5, 7, 10, 2, 3, 20, 12], outside=((50, 7), (300,)))
    assert_attention_close(run(s, always=False), prefill64(s), "outside")


def test_a_bound_below_the_longest_sequence_keeps_the_others_right():
    s = make([(200, [230, 300, 215])], 8, 2, 128, 16, seed=780, new=[20, 64, 5])
    want = prefill64(s)
    out = run(s, max_q_len=32)  # rows of the second sequence past the grid hold anything
    rows = [*range(20), *range(84, 89)]
    assert_attention_close(out[rows], want[rows], "the others")


def test_two_calls_at_once_on_two_streams():
    cases = [make([(2000, [2010 + 3 * i for i in range(12)])], 8, 2, 128, 16, seed=781,
                  new=[1 + i % 9 for i in range(12)]),
             make([(700, [800, 705, 1000])], 16, 2, 128, 32, seed=782, new=[90, 5, 250])]
    want = [run(s) for s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream, out in zip(cases, streams, outs):
            with torch.cuda.stream(stream):
                out.append(pa.prefill_shared(s.q, s.k_cache, s.v_cache, s.bt, s.cu_q, s.cu_k,
                                             s.cu_groups, s.prefix_lens, s.scale, always=True,
                                             max_q_len=max(s.new)))
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    for w, out in zip(want, outs):
        assert all(torch.equal(w, o) for o in out)


def test_a_workspace_for_the_most_rows_and_groups_serves_fewer():
    kc = torch.zeros((4, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    for H, rows in ((32, [1, 32, 33, 64, 65, 960, 961, 100000]), (128, [8, 9, 16, 17, 4000]),
                    (8, [1, 128, 129, 257])):
        need = torch.tensor([[pa.prefill_shared_workspace_size(kc, t, H, g)
                              for g in (0, 1, 2, 3, 16, 30, 31, 500, 16384)] for t in rows])
        assert (need > 0).all()
        assert (need.diff(dim=0) >= 0).all() and (need.diff(dim=1) >= 0).all(), need
    s = make([(200, [230 + i for i in range(32)])], 32, 8, 128, 16, seed=783, new=[30] * 32)
    want = prefill64(s)
    ws = torch.full((pa.prefill_shared_workspace_size(s.k_cache, 960, 32, 30),), 255,
                    dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for cu in ([*range(0, 60, 2)][:16] + [32], [0, 32], [*range(30)] + [32]):
        s.cu_groups, s.prefix_lens = i32(cu), i32([200] * (len(cu) - 1))
        assert_attention_close(run(s, workspace=ws), want, f"groups {cu}")


@pytest.mark.parametrize("new, prefix", [([200, 256, 130], 600), ([3] * 40, 6000)])
def test_always_where_the_choice_is_measured(new, prefix):
    # the rows of test_without_always_calls_that_would_not_gain_are_prefill against 64 bits; the first
    # form has a team of lanes for each row in its merge
    s = make([(prefix, [prefix + n + 9 for n in new])], 32, 8, 128, 16, seed=760, new=new)
    want = prefill64(s)
    assert_attention_close(run(s), want, "always")
    assert_attention_close(run(s, always=False), want, "chosen")


@pytest.mark.parametrize("groups", [513, 1025])
def test_more_groups_than_fit_the_plan_or_one_of_its_passes(groups):
    # one prefix for all sequences: any partition of them is one of groups that share it
    r = np.random.default_rng(groups)
    n = 700
    new = [int(x) for x in r.integers(0, 4, n)]
    s = make([(50, [max(k, 49 + int(x)) for k, x in zip(new, r.integers(0, 40, n))])], 2, 1, 128, 16,
             seed=784, new=new)
    cu = np.sort(r.integers(0, n + 1, groups + 1))
    at = r.integers(0, groups + 1, groups // 5)
    cu[at] = r.integers(-50, n, len(at))
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    s.cu_groups, s.prefix_lens = i32(cu), i32(r.integers(-5, 51, groups))
    want = prefill64(s)
    assert_attention_close(run(s), want, f"{groups} groups")
    assert_attention_close(run(s, always=False), want, f"{groups} groups, chosen")


@pytest.mark.parametrize("where", ["own", "shared", "both"])
@pytest.mark.parametrize("new", [[1 + i % 5 for i in range(40)], [70, 33, 64, 130, 1, 90]])
def test_weights_of_few_dominant_keys_keep_more_bits_than_bf16(where, new):
    # q of a kv head's heads is one direction and a little noise, three keys of the prefix or of each
    # sequence's own lie along it: their scores are near 11, those of the 600 others N(0, 1), so they
    # hold 98 % of the weight. An output is then off by at most
    #   own keys: the scores' fp32 error (below 2^-12 of a weight in all) and 2^-16 of a weight, the
    #             second of P's two bf16 terms rounding what the first left, both by 2^-8; with 2 % of
    #             the weight on keys of the other kind
    #   shared keys: 2^-11 of a weight (f16) instead
    # of the largest |V|, and twice that beyond the rounding of the exact result where the output
    # rounds to the other side of it. One bf16 term would be off by 2^-8 of a weight.
    weights_of_few_keys_hold(where, new, run, prefill64)


def weights_of_few_keys_hold(where, new, call, definition):
    n = len(new)
    s = make([(200, [600 + x + 7 * (i % 9) for i, x in enumerate(new)])], 8, 2, 128, 16, seed=785, new=new)
    g = torch.Generator().manual_seed(786)
    base = torch.randn((2, 128), generator=g)
    q = base.repeat_interleave(4, dim=0) + 0.25 * torch.randn(s.q.shape, generator=g)
    s.q.copy_(q.to(torch.bfloat16))
    bt = s.bt.cpu()
    spots = {(bt[b, p // 16].item(), p % 16) for b in range(n)
             for p in {"own": (195, 340, 530), "shared": (3, 100, 188), "both": (3, 195, 530)}[where]}
    for block, at in sorted(spots):
        s.k_cache[block, at] = (base + 0.15 * torch.randn((2, 128), generator=g)).to(torch.bfloat16).cuda()
    want = definition(s)
    got = n64(call(s))
    bits = 2.0 ** -12 + (2.0 ** -16 + 0.02 * 2.0 ** -11 if where == "own" else 2.0 ** -11)
    top = np.abs(n64(s.v_cache)).max()
    rounding = np.abs(n64(torch.from_numpy(want).float().to(torch.bfloat16)) - want)
    assert (np.abs(got - want) - rounding).max() <= 2 * bits * top
