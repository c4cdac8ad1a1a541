"""pa_prefill_window against a plain 64-bit implementation, with the attention
tolerance of the library (bf16 output, fp32 accumulation), and against
pa_prefill_varlen where the window keeps every key."""
import numpy as np
import pytest
import torch

import ops64
import paged_kv_cache_186_gb300 as pa
import workloads as W
from gpu_util import assert_attention_close, to_device

pytestmark = pytest.mark.gpu


def case_inputs(H, Hkv, bs, cached, q_lens, seed):
    h = W.make_prefill(len(q_lens), H, Hkv, 128, bs, cached, q_lens, seed=seed)
    g = to_device(h)
    pa.store_kv(g.k_new, g.v_new, g.slot_mapping, g.k_cache, g.v_cache)
    torch.cuda.synchronize()
    return g


def want64(g, window, sinks):
    n64 = lambda t: t.float().cpu().double().numpy()
    return ops64.prefill_window(n64(g.q), n64(g.k_cache), n64(g.v_cache),
                                g.block_tables.cpu().numpy(), g.cu_seqlens_q.cpu().numpy(),
                                g.cu_seqlens_k.cpu().numpy(), g.scale, window, sinks)


def run(g, window, sinks, max_q_len=0):
    out = pa.prefill_window(g.q, g.k_cache, g.v_cache, g.block_tables, g.cu_seqlens_q,
                            g.cu_seqlens_k, g.scale, window, sinks, max_q_len=max_q_len)
    torch.cuda.synchronize()
    assert pa.get_device_error() == 0
    return out


def poison_unseen(g, window, sinks, bs, cut_table=True):
    """NaN in K and V of every key no row of the call sees; table entries of blocks that hold
    only such keys become -1 (freed)."""
    cu_q, cu_k = g.cu_seqlens_q.cpu().numpy(), g.cu_seqlens_k.cpu().numpy()
    bt = g.block_tables.cpu().numpy().copy()
    for b in range(len(cu_q) - 1):
        n, kv = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        lo = max(0, kv - n - window + 1) if n else kv
        for j in range(min(sinks if n else 0, lo), lo):
            g.k_cache[bt[b, j // bs], j % bs] = float("nan")
            g.v_cache[bt[b, j // bs], j % bs] = float("nan")
        for j in range(kv, -(-kv // bs) * bs):  # behind the last key
            g.k_cache[bt[b, j // bs], j % bs] = float("nan")
            g.v_cache[bt[b, j // bs], j % bs] = float("nan")
        if cut_table:
            first = -(-min(sinks if n else 0, lo) // bs)
            g.block_tables[b, first:lo // bs] = -1


SHAPES = [
    # H, Hkv, bs, cached, q_lens
    (4, 1, 16, [40], [32]),
    (32, 8, 16, [0, 100, 700, 7], [128, 300, 129, 200]),
    (8, 2, 32, [5, 1000], [1, 255]),
    (4, 4, 16, [64, 0, 300], [33, 17, 1]),       # group 1
    (8, 4, 16, [300], [200]),                    # group 2
    (16, 2, 32, [128, 900], [256, 65]),          # group 8
    (16, 1, 16, [17, 500], [40, 3]),             # group 16
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: f"H{c[0]}kv{c[1]}bs{c[2]}n{len(c[4])}")
@pytest.mark.parametrize("window, sinks", [(1, 0), (2, 1), (17, 4), (64, 0), (100, 28), (128, 4),
                                           (129, 130), (200, 300), (513, 64), (5000, 4)])
def test_matches_64_bits_with_unseen_keys_poisoned(shape, window, sinks):
    H, Hkv, bs, cached, q_lens = shape
    g = case_inputs(H, Hkv, bs, cached, q_lens, seed=90 + H + window)
    want = want64(g, window, sinks)
    poison_unseen(g, window, sinks, bs)
    assert_attention_close(run(g, window, sinks, max(q_lens)), want, f"{shape} {window} {sinks}")


def test_a_window_over_every_key_is_prefill_varlen():
    g = case_inputs(32, 8, 16, [0, 333, 90], [400, 65, 1], seed=120)
    full = pa.prefill_varlen(g.q, g.k_cache, g.v_cache, g.block_tables, g.cu_seqlens_q,
                             g.cu_seqlens_k, g.scale)
    for window, sinks in ((400, 0), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        out = run(g, window, sinks)
        # the same keys in the same tiles; P may be rounded in other places
        assert (out.float() - full.float()).abs().max().item() <= 2e-2
        assert_attention_close(out, want64(g, window, sinks), str(window))


def test_long_prompt_with_a_small_window():
    g = case_inputs(8, 2, 16, [0, 3000], [2500, 40], seed=121)
    for window, sinks in ((256, 4), (1000, 200)):
        want = want64(g, window, sinks)
        assert_attention_close(run(g, window, sinks), want, f"{window} {sinks}")


def test_empty_sequences_and_rows_behind_the_last_one():
    g = case_inputs(8, 2, 16, [10, 50, 0, 20], [5, 0, 0, 37], seed=122)
    want = want64(g, 16, 2)
    T = g.q.shape[0]
    out = torch.full((T, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    pa.prefill_window(g.q, g.k_cache, g.v_cache, g.block_tables, g.cu_seqlens_q, g.cu_seqlens_k,
                      g.scale, 16, 2, out=out)
    assert_attention_close(out, want, "empty sequences")
    # a longer packed buffer: rows past cu_seqlens_q[batch] stay as they were
    q = torch.cat([g.q, torch.full((9, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full((T + 9, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    pa.prefill_window(q, g.k_cache, g.v_cache, g.block_tables, g.cu_seqlens_q, g.cu_seqlens_k,
                      g.scale, 16, 2, out=out)
    torch.cuda.synchronize()
    assert (out[T:] == 3.0).all()
    assert_attention_close(out[:T], want, "padded buffer")


def test_more_queries_than_keys_gives_zero_rows_where_nothing_is_seen():
    # invalid lengths (q_len > kv_len): keys are clamped, rows past them see only what their
    # window still reaches
    g = case_inputs(4, 1, 16, [0], [100], seed=123)
    g.cu_seqlens_k[1] = 20
    for window, sinks in ((8, 0), (8, 3), (50, 0)):
        out = run(g, window, sinks)
        want = want64(g, window, sinks)
        # want64 takes cached = 0 as the call does
        assert_attention_close(out, want, f"{window} {sinks}")
        if sinks == 0:
            assert (out[20 + window:] == 0).all()


def test_block_ids_out_of_range_are_flagged():
    g = case_inputs(4, 1, 16, [100], [16], seed=124)
    g.block_tables[0, 6] = g.k_cache.shape[0]  # inside the window
    pa.prefill_window(g.q, g.k_cache, g.v_cache, g.block_tables, g.cu_seqlens_q, g.cu_seqlens_k,
                      g.scale, 64, 0)
    assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_RANGE
    g.block_tables[0, 1] = -7  # outside of it: not read
    g.block_tables[0, 6] = 0
    run(g, 64, 0)


def test_strided_q_and_graph_replay():
    g = case_inputs(8, 2, 16, [200, 5], [30, 60], seed=125)
    big = torch.zeros((90, 12, 128), dtype=torch.bfloat16, device="cuda")
    big[:, 2:10] = g.q
    want = want64(g, 48, 4)
    out = pa.prefill_window(big[:, 2:10], g.k_cache, g.v_cache, g.block_tables, g.cu_seqlens_q,
                            g.cu_seqlens_k, g.scale, 48, 4)
    assert_attention_close(out, want, "strided q")
    res = torch.zeros_like(out)
    run(g, 48, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.prefill_window(g.q, g.k_cache, g.v_cache, g.block_tables, g.cu_seqlens_q,
                          g.cu_seqlens_k, g.scale, 48, 4, out=res)
    for k in range(2):
        g.q.copy_(torch.randn_like(g.q))
        graph.replay()
        torch.cuda.synchronize()
        assert_attention_close(res, want64(g, 48, 4), f"replay {k}")


@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("window, sinks", [(1, 0), (60, 70), (130, 4), (700, 0), (4000, 40)])
def test_one_query_tile_a_sequence(group, bs, window, sinks):
    # one to a dozen key tiles, shared in turn by the halves of a CTA
    most = 128 // group
    q_lens = [1, most, max(1, most // 2), 1, most, 0, min(3, most)]
    cached = [0, 0, 127, 128, 260, 33, 1500]
    g = case_inputs(2 * group, 2, bs, cached, q_lens, seed=130 + group + bs + window)
    want = want64(g, window, sinks)
    poison_unseen(g, window, sinks, bs)
    assert_attention_close(run(g, window, sinks, most), want, f"{group} {bs} {window} {sinks}")


def test_short_sequences_repeat_bit_for_bit():
    # one query tile a sequence, the walked tiles shared by the CTA's halves: back-to-back
    # launches over many key tiles, and ring stages used by both halves in turn
    g = case_inputs(8, 2, 16, [3000, 700, 5, 1234, 0], [1, 32, 7, 16, 9], seed=126)
    first = run(g, 2000, 4, max_q_len=32)
    assert_attention_close(first, want64(g, 2000, 4), "short sequences")
    out = torch.empty_like(first)
    for _ in range(20):
        for _ in range(50):
            pa.prefill_window(g.q, g.k_cache, g.v_cache, g.block_tables, g.cu_seqlens_q,
                              g.cu_seqlens_k, g.scale, 2000, 4, max_q_len=32, out=out)
        assert torch.equal(out, first)
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("group, bs", [(4, 16), (1, 32), (16, 16), (8, 32)])
@pytest.mark.parametrize("window, sinks", [(20, 4), (130, 0), (1000, 4), (60, 300)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_later_tokens_in_a_pairs_last_block_may_hold_anything(group, bs, window, sinks, bad):
    # the last block a pair of query tiles sees also holds the next pair's first keys: K and V
    # there reach no row of the pairs before
    pair = 2 * (128 // group)
    g = case_inputs(group, 1, bs, [5], [3 * pair + 7], seed=140 + group + window)
    want = want64(g, window, sinks)
    bt = g.block_tables.cpu().numpy()
    clean = g.k_cache.clone(), g.v_cache.clone()
    for k in (1, 2, 3):
        end = 5 + k * pair  # keys of the pairs before the k-th
        assert end % bs
        for j in range(end, -(-end // bs) * bs):
            g.k_cache[bt[0, j // bs], j % bs] = bad
            g.v_cache[bt[0, j // bs], j % bs] = bad
        rows = k * pair
        assert_attention_close(run(g, window, sinks)[:rows], want[:rows], f"{k} {bad}")
        g.k_cache.copy_(clean[0])
        g.v_cache.copy_(clean[1])


@pytest.mark.parametrize("cached, q_lens", [([300, 0, 700], [70, 200, 1]),  # two query tiles a CTA
                                            ([300, 129, 2000], [32, 20, 1])])  # one
@pytest.mark.parametrize("window, sinks", [(200, 4), (1000, 4), (300, 128), (5000, 1)])
def test_rows_whose_weight_lies_on_the_sinks(cached, q_lens, window, sinks):
    """Four sinks hold nearly all the weight, in proportions that differ from row to row.

    Only the first dim of q and K is not zero, so every score is one exact product. Of the
    weights, exp2's argument (below 8 where the weight counts: 2 roundings of 2^-24 * 8, times
    ln 2) and ex2.approx (2^-22) give 2^-20, two bf16 terms 2^-17; the fp32 sums of at most a few
    hundred terms 2^-16 each: together below 2^-14 of sum w |v|, next to the output's own
    rounding, 2^-8 of it. With the weights rounded once to bf16 an output would be off by up to
    2^-9 of sum w |v|, thirty times as much."""
    g = case_inputs(8, 2, 16, cached, q_lens, seed=150 + window + sinks)
    gen = torch.Generator().manual_seed(151)
    bt = g.block_tables.cpu().numpy()
    g.k_cache.zero_()
    g.k_cache[..., 0] = -40.0
    for b in range(len(q_lens)):
        g.k_cache[bt[b, 0], :4, :, 0] = -torch.rand((4, 2), generator=gen).to(torch.bfloat16).cuda()
    q0 = (0.5 + 1.5 * torch.rand(g.q.shape[:2], generator=gen)).to(torch.bfloat16).cuda()
    g.q.zero_()
    g.q[..., 0] = q0
    g.scale = 1.0
    want = want64(g, window, sinks)
    v = g.v_cache.clone()
    g.v_cache.abs_()
    mag = want64(g, window, sinks)
    g.v_cache.copy_(v)
    got = run(g, window, sinks, max(q_lens)).float().cpu().double().numpy()
    over = np.abs(got - want) - (np.abs(want) * 2.0 ** -8 + mag * 2.0 ** -14)
    assert over.max() <= 0, f"{float(over.max()):.3e} past the bound"
