"""pa_evict against a sort of every head's middle keys: exact (copies and indexes)."""
import numpy as np
import pytest
import torch

import ops64
import paged_kv_cache_186_gb300 as pa
import workloads as W

pytestmark = pytest.mark.gpu


def make(lens, Hkv, D, bs, kv="bf16", seed=0, extra_cols=1):
    gen = torch.Generator().manual_seed(seed)
    need = [max(1, -(-n // bs)) for n in lens]
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=gen).to(torch.int32)
    bt = torch.full((len(lens), max(need) + extra_cols), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        bt[i, :n] = perm[at:at + n]
        at += n
    s = dict(lens=lens, bs=bs, bt=bt)
    shape = (nb, bs, Hkv, D)
    if kv == "bf16":
        s["kc"], s["vc"] = (torch.randn(shape, generator=gen).to(torch.bfloat16) for _ in range(2))
        s["ks"] = s["vs"] = None
    else:
        dt = torch.uint8 if kv == "fp8" else torch.int8
        s["kc"], s["vc"] = (torch.randint(0, 120, shape, generator=gen).to(dt) for _ in range(2))
        s["ks"], s["vs"] = (torch.rand((nb, Hkv, bs), generator=gen) for _ in range(2))
    s["scores"] = torch.rand((nb, Hkv, bs), generator=gen)
    return s


def run(s, budget, sinks=0, recent=0, **kw):
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    lens = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    new, kept = pa.evict(dev["kc"], dev["vc"], dev["scores"], dev["bt"], lens, budget, sinks=sinks,
                         recent=recent, k_scale=dev["ks"], v_scale=dev["vs"], **kw)
    torch.cuda.synchronize()
    return dev, new, kept


def same_bits(a, b):
    as_int = {2: torch.int16, 4: torch.int32, 1: torch.uint8}
    a, b = a.cpu(), b.cpu()
    return torch.equal(a.view(as_int[a.element_size()]), b.view(as_int[b.element_size()]))


def check(s, budget, sinks=0, recent=0, lens=None, **kw):
    dev, new, kept = run(s, budget, sinks, recent, **kw)
    assert pa.get_device_error() == 0
    lens = s["lens"] if lens is None else lens
    bt = s["bt"].numpy()
    want, wlens = ops64.evict_rows(s["scores"].numpy(), bt, lens, budget, sinks, recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(new.cpu().numpy(), wlens)
    for name, by_slot in (("kc", True), ("vc", True), ("scores", False), ("ks", False),
                          ("vs", False)):
        if s[name] is not None:
            moved = ops64.move_rows(s[name], by_slot, want, bt, lens, budget, s["bs"])
            assert same_bits(dev[name], moved), name
    return dev, new, kept


CASES = [
    # lens, Hkv, D, bs, kv, budget, sinks, recent
    ([1], 1, 64, 16, "bf16", 1, 0, 0),
    ([2], 1, 64, 16, "bf16", 1, 0, 0),
    ([2, 5, 0], 2, 64, 16, "bf16", 1, 1, 0),
    ([40, 0, 17, 16, 100], 2, 64, 16, "bf16", 16, 2, 4),
    ([40, 33, 100], 3, 128, 32, "bf16", 33, 0, 33),      # recent only
    ([40, 33, 100], 3, 128, 32, "bf16", 33, 33, 0),      # sinks only
    ([40, 33, 100], 1, 128, 16, "bf16", 33, 10, 23),     # nothing by score
    ([300, 301, 5], 2, 128, 16, "fp8", 100, 4, 31),
    ([300, 64, 65], 4, 128, 32, "fp8", 64, 0, 0),
    ([700, 10], 2, 128, 16, "int8", 513, 4, 100),
    ([1500, 1023, 1024, 1025], 2, 128, 16, "bf16", 1024, 4, 256),
    ([5000, 3000], 1, 64, 32, "bf16", 2000, 0, 1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"L{max(c[0])}kv{c[1]}D{c[2]}bs{c[3]}{c[4]}b{c[5]}")
def test_matches_the_sort(case):
    lens, Hkv, D, bs, kv, budget, sinks, recent = case
    check(make(lens, Hkv, D, bs, kv, seed=len(lens) + budget), budget, sinks, recent)


def test_ties_go_to_the_lowest_position():
    s = make([500, 130], 2, 64, 16, seed=300)
    s["scores"] = torch.floor(s["scores"] * 4)  # four distinct values
    for budget in (1, 17, 100, 129):
        check(s, budget, 2 if budget > 4 else 0, budget // 4)
    s["scores"].zero_()  # all equal, both zeros
    s["scores"][:, :, ::2] = -0.0
    _, _, kept = check(s, 50, 0, 10)
    assert kept[0, 0, :40].tolist() == list(range(40))


def test_special_values():
    s = make([400, 90], 2, 64, 16, seed=301)
    gen = torch.Generator().manual_seed(1)
    r = torch.randint(0, 12, s["scores"].shape, generator=gen)
    sp = [float("nan"), float("inf"), -float("inf"), -0.0, 0.0, 1e-42, -1e-42, 3.4e38, -3.4e38]
    for i, v in enumerate(sp):
        s["scores"][r == i] = v
    s["scores"][r == 9] *= -1.0
    for budget in (5, 30, 60, 88, 300):
        check(s, budget, 1, 2)


def test_every_nan_is_the_largest_whatever_its_bits():
    s = make([300], 2, 64, 16, seed=309)
    bits = s["scores"].view(torch.int32)
    gen = torch.Generator().manual_seed(3)
    r = torch.randint(0, 8, bits.shape, generator=gen)
    for i, pattern in enumerate((0x7fc00000, -0x400000, 0x7f800001, -1, 0x7fffffff)):
        bits[r == i] = pattern  # quiet and signalling, both signs
    for budget in (10, 150, 250):
        check(s, budget)


def test_scores_that_differ_in_the_last_bits_only():
    s = make([600], 1, 64, 16, seed=302)
    bits = 0x3f800000 + torch.randint(0, 40, s["scores"].shape,
                                      generator=torch.Generator().manual_seed(2))
    s["scores"] = bits.to(torch.int32).view(torch.float32)
    for budget in (3, 100, 599):
        check(s, budget)


@pytest.mark.parametrize("seed", range(12))
def test_random_cases(seed):
    r = np.random.RandomState(seed)
    kv = ["bf16", "fp8", "int8"][r.randint(3)]
    D = 128 if kv != "bf16" else [64, 128][r.randint(2)]
    bs = [16, 32][r.randint(2)]
    lens = [int(x) for x in np.exp(r.uniform(0, 7.5, size=r.randint(1, 7)))]
    budget = int(np.exp(r.uniform(0, 6.5)))
    sinks = r.randint(0, min(budget, 8) + 1)
    recent = r.randint(0, budget - sinks + 1)
    check(make(lens, r.randint(1, 5), D, bs, kv, seed=seed), budget, sinks, recent)


def test_a_long_sequence():
    s = make([60000], 1, 64, 32, seed=303)
    check(s, 3000, 4, 100)


@pytest.mark.parametrize("lens, budget", [([9000, 16384, 5], 2000), ([33000, 8192], 500),
                                          ([100000], 4096)])
def test_clusters_of_every_size_and_keys_that_are_not_held(lens, budget):
    check(make(lens, 1, 64, 16, seed=len(lens) + budget), budget, 3, 40)


@pytest.mark.parametrize("lens", [[6000], [20000, 12001], [90000]])
def test_more_equal_keys_than_a_warp_lists(lens):
    s = make(lens, 1, 64, 32, seed=311)
    s["scores"][:] = 2.5
    check(s, 1500, 2, 30)
    gen = torch.Generator().manual_seed(5)
    # one bin of the first digit, then a few values far below it
    s["scores"] = 1.0 + torch.rand(s["scores"].shape, generator=gen) * 2.0 ** -4
    s["scores"][torch.rand(s["scores"].shape, generator=gen) < 0.1] = 1e-20
    check(s, 1500, 2, 30)
    check(s, min(lens) - 3, 0, 0)


def test_length_bound_and_capacity_clamp_the_lengths():
    s = make([100, 50], 2, 64, 16, seed=304)
    check(s, 20, 2, 5, lens=[60, 50], max_context_len=60)
    cap = dict(s, bt=s["bt"][:, :4].contiguous())  # table of 64 positions
    check(cap, 20, 2, 5, lens=[64, 50])


def test_block_ids_out_of_range_are_flagged():
    s = make([100, 40], 2, 64, 16, seed=305)
    s["bt"][0, 3] = -1
    s["bt"][0, 5] = s["kc"].shape[0] + 7
    dev, new, kept = run(s, 32, 0, 8)
    assert pa.get_device_error() == pa.PA_DEVERR_BLOCK_RANGE
    assert new.tolist() == [32, 32]
    assert kept.min() >= 0 and kept.max() < 100
    # the other sequence is right
    want, _ = ops64.evict_rows(s["scores"].numpy(), s["bt"].numpy().clip(0, s["kc"].shape[0] - 1),
                               [100, 40], 32, 0, 8)
    assert np.array_equal(kept[1].cpu().numpy(), want[1])


def test_other_stream_graph_replay_and_given_outputs():
    s = make([90, 300], 2, 128, 16, seed=306)
    want, wlens = ops64.evict_rows(s["scores"].numpy(), s["bt"].numpy(), s["lens"], 64, 2, 16)
    kept = torch.zeros((2, 2, 64), dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(s, 64, 2, 16, kept=kept, new_lens=new)
    assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(new.cpu().numpy(), wlens)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    lens = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.evict(dev["kc"], dev["vc"], dev["scores"], dev["bt"], lens, 64, sinks=2, recent=16,
                 kept=kept, new_lens=new)
    for k in range(2):
        for n in ("kc", "vc", "scores"):
            dev[n].copy_(torch.randn_like(dev[n]))
        t = {n: dev[n].cpu() for n in ("kc", "vc", "scores")}
        graph.replay()
        torch.cuda.synchronize()
        want, _ = ops64.evict_rows(t["scores"].numpy(), s["bt"].numpy(), s["lens"], 64, 2, 16)
        assert np.array_equal(kept.cpu().numpy(), want)
        for n, by_slot in (("kc", True), ("vc", True), ("scores", False)):
            assert same_bits(dev[n], ops64.move_rows(t[n], by_slot, want, s["bt"].numpy(),
                                                     s["lens"], 64, 16))


def test_strided_tables_and_lengths_are_taken():
    s = make([90, 30], 2, 64, 16, seed=310)
    want, _ = ops64.evict_rows(s["scores"].numpy(), s["bt"].numpy(), s["lens"], 20, 0, 4)
    wide = torch.full((2, s["bt"].shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :s["bt"].shape[1]] = s["bt"].cuda()
    lens = torch.tensor([[90, 1], [30, 1]], dtype=torch.int32, device="cuda")
    _, kept = pa.evict(s["kc"].cuda(), s["vc"].cuda(), s["scores"].cuda(),
                       wide[:, :s["bt"].shape[1]], lens[:, 0], 20, recent=4)
    assert np.array_equal(kept.cpu().numpy(), want)


def test_decode_after_evict_sees_the_new_lengths_and_rows():
    # evict directly before a decode that takes its new_lens, repeatedly
    h = W.make_decode(4, 8, 2, 128, 16, [100, 300, 20, 64], seed=307)
    for seed in range(5):
        s = make([100, 300, 20, 64], 2, 128, 16, seed=308 + seed)
        dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
        lens = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
        q = h.q.cuda()
        new = torch.full((4,), 1, dtype=torch.int32, device="cuda")
        kept = torch.zeros((4, 2, 64), dtype=torch.int32, device="cuda")
        pa.evict(dev["kc"], dev["vc"], dev["scores"], dev["bt"], lens, 64, recent=8, kept=kept,
                 new_lens=new)
        out = pa.decode(q, dev["kc"], dev["vc"], dev["bt"], new, 0.1)
        torch.cuda.synchronize()
        again = pa.decode(q, dev["kc"], dev["vc"], dev["bt"],
                          torch.tensor([64, 64, 20, 64], dtype=torch.int32, device="cuda"), 0.1)
        assert torch.equal(out, again)
