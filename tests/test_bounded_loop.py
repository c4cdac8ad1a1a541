"""The bounded-cache operators together: a prompt (norm_rope_store, prefill_window), then
decode steps (norm_rope_store, decode_scored) with an evict every few of them, against the
same loop in plain 64-bit arithmetic on the caches the library wrote."""
import numpy as np
import pytest
import torch

import ops64
import paged_kv_cache_186_gb300 as pa
from gpu_util import assert_attention_close
from test_norm_rope import check_rows, table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_generation_over_a_bounded_cache(kv):
    H, Hkv, D, bs, B = 8, 2, 128, 16, 3
    prompts, budget, sinks, recent, every, steps = [70, 5, 41], 48, 2, 16, 6, 30
    g = torch.Generator().manual_seed(400)
    nb, width = 64, 10
    bt = torch.randperm(nb, generator=g)[:B * width].view(B, width).to(torch.int32).cuda()
    if kv == "bf16":
        kc, vc = (torch.full((nb, bs, Hkv, D), float("nan"), dtype=torch.bfloat16).cuda()
                  for _ in range(2))
        ks = vs = None
    else:
        kc, vc = (torch.full((nb, bs, Hkv, D), 0x7f, dtype=torch.uint8).cuda() for _ in range(2))
        ks, vs = (torch.full((nb, Hkv, bs), float("nan")).cuda() for _ in range(2))
    scores = torch.full((nb, Hkv, bs), float("nan")).cuda()
    cs = torch.from_numpy(table(512, D)).cuda()
    qw, kw = (1 + 0.2 * torch.randn((2, D), generator=g)).to(torch.bfloat16).cuda()
    scale = 1 / np.sqrt(D)
    n64 = lambda t: t.float().cpu().double().numpy()

    def store(n_per_seq, slot_pos, pos):
        """Project, norm, rotate and store new tokens; slots from cache positions slot_pos."""
        T = sum(n_per_seq)
        qkv = torch.randn((T, (H + 2 * Hkv) * D), generator=g).to(torch.bfloat16).cuda()
        q, k, v = (x.view(T, -1, D) for x in qkv.split([H * D, Hkv * D, Hkv * D], dim=1))
        rows = bt.cpu().numpy()
        slots, at = [], 0
        for b, n in enumerate(n_per_seq):
            for p in slot_pos[at:at + n]:
                slots.append(int(rows[b, p // bs]) * bs + p % bs)
            at += n
        out = pa.norm_rope_store(q, k, v, torch.tensor(pos).cuda(), torch.tensor(slots).cuda(), kc,
                                 vc, q_weight=qw, k_weight=kw, cos_sin=cs, k_scale=ks, v_scale=vs,
                                 scores=scores)
        want, mag = ops64.norm_rope(n64(q), n64(qw), 1e-6, cs.cpu().numpy(), np.array(pos), False)
        check_rows(n64(out), want, mag, "q")
        return out

    def values():
        return (ops64.cache_values(c.cpu(), None if s is None else s.cpu())
                for c, s in ((kc, ks), (vc, vs)))

    where = [p for n in prompts for p in range(n)]
    q = store(prompts, where, where)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32).cuda()
    if kv == "bf16":
        out = pa.prefill_window(q, kc, vc, bt, cu, cu, scale, 32, sinks)
        K, V = values()
        want = ops64.prefill_window(n64(q), np.nan_to_num(K), np.nan_to_num(V), bt.cpu().numpy(),
                                    cu.cpu().numpy(), cu.cpu().numpy(), scale, 32, sinks)
        assert_attention_close(out, want, "prompt")
    lens = torch.tensor(prompts, dtype=torch.int32).cuda()
    position = list(prompts)  # a token's position keeps counting past evictions
    cut = 0
    for step in range(steps):
        host = lens.tolist()
        q = store([1] * B, host, position)
        position = [p + 1 for p in position]
        lens = lens + 1
        before = n64(scores)
        out = pa.decode_scored(q, kc, vc, bt, lens, scores, scale, k_scale=ks, v_scale=vs)
        K, V = values()
        want, add, mag = ops64.decode_scored(n64(q), np.nan_to_num(K), np.nan_to_num(V),
                                             bt.cpu().numpy(), lens.tolist(), scale,
                                             tuple(scores.shape))
        assert_attention_close(out, want, f"step {step}")
        live = add > 0
        tol = mag * 2.0 ** -15 + add * 2.0 ** -19 + np.abs(before) * 2.0 ** -23
        assert (np.abs(n64(scores) - before - add)[live] <= tol[live]).all()
        if step % every == every - 1:
            s = {n: t.cpu() if t is not None else None
                 for n, t in (("kc", kc), ("vc", vc), ("scores", scores), ("ks", ks), ("vs", vs))}
            lens, kept = pa.evict(kc, vc, scores, bt, lens, budget, sinks=sinks, recent=recent,
                                  k_scale=ks, v_scale=vs)
            host = [n + 1 for n in host]
            rows, new = ops64.evict_rows(s["scores"].numpy(), bt.cpu().numpy(), host, budget, sinks,
                                         recent)
            assert np.array_equal(kept.cpu().numpy(), rows)
            assert np.array_equal(lens.cpu().numpy(), new)
            for n, t, by_slot in (("kc", kc, True), ("vc", vc, True), ("scores", scores, False)):
                moved = ops64.move_rows(s[n], by_slot, rows, bt.cpu().numpy(), host, budget, bs)
                bits = torch.uint8 if by_slot and kv == "fp8" else torch.int16 if by_slot else torch.int32
                assert torch.equal(t.cpu().view(bits), moved.view(bits)), n
            cut += int((np.array(host) > budget).sum())
    assert pa.get_device_error() == 0
    assert cut >= 5 and lens.max() <= budget + every


def test_empty_calls_change_nothing():
    kc, vc = (torch.ones((4, 16, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    scores = torch.ones((4, 2, 16), device="cuda")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64, device="cuda")
    assert pa.norm_rope_store(bf(0, 4, 128), bf(0, 2, 128), bf(0, 2, 128), i64(0), i64(0), kc, vc,
                              cos_sin=torch.ones((3, 64), device="cuda"),
                              scores=scores).shape == (0, 4, 128)
    assert pa.prefill_window(bf(0, 4, 128), kc, vc, i32(2, 1), i32(3), i32(3), 0.1, 8).numel() == 0
    assert pa.prefill_window(bf(0, 4, 128), kc, vc, i32(0, 1), i32(1), i32(1), 0.1, 8).numel() == 0
    assert pa.decode_scored(bf(0, 4, 128), kc, vc, i32(0, 1), i32(0), scores, 0.1).numel() == 0
    new, kept = pa.evict(kc, vc, scores, i32(0, 1), i32(0), 8)
    assert new.numel() == 0 and kept.shape == (0, 2, 8)
    out = pa.decode_scored(bf(2, 4, 128) + 1, kc, vc, i32(2, 1), i32(2), scores, 0.1)
    new, kept = pa.evict(kc, vc, scores, i32(2, 1), i32(2), 8, sinks=1, recent=2)
    torch.cuda.synchronize()
    assert (out == 0).all() and (new == 0).all() and (kept == -1).all()
    assert (kc == 1).all() and (vc == 1).all() and (scores == 1).all()
    assert pa.get_device_error() == 0


def test_lengths_written_right_before_a_store_and_a_decode():
    # a torch kernel raises the lengths, norm_rope_store follows it, then a decode that reads
    # the lengths before its own dependency wait: every step sees that step's lengths
    g = torch.Generator().manual_seed(401)
    B, H, Hkv, D, bs, width = 16, 8, 2, 128, 16, 30
    kc, vc = (torch.randn((B * width, bs, Hkv, D), generator=g).to(torch.bfloat16).cuda()
              for _ in range(2))
    bt = torch.randperm(B * width, generator=g).view(B, width).to(torch.int32).cuda()
    lens = torch.randint(1, 200, (B,), generator=g).to(torch.int32).cuda()
    start = lens.clone()
    steps = 200
    qkv = torch.randn((steps, B, H + 2 * Hkv, D), generator=g).to(torch.bfloat16).cuda()
    rows = torch.arange(B, device="cuda")
    slots = []
    for s in range(steps):
        p = (start + s).long()
        slots.append(bt[rows, p // bs].long() * bs + p % bs)
    outs = torch.zeros((steps, B, H, D), dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros((B * width, Hkv, bs), device="cuda")
    ws = torch.empty(pa.decode_scored_workspace_size(kc, B, H, width), dtype=torch.uint8,
                     device="cuda")
    first = kc.clone(), vc.clone()
    torch.cuda.synchronize()
    for s in range(steps):
        x = qkv[s]
        lens.add_(1)
        q = pa.norm_rope_store(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], None, slots[s], kc, vc)
        if s % 2:
            pa.decode_scored(q, kc, vc, bt, lens, scores, 0.1, out=outs[s], workspace=ws)
        else:
            pa.decode(q, kc, vc, bt, lens, 0.1, out=outs[s], workspace=ws)
    torch.cuda.synchronize()
    kc.copy_(first[0])
    vc.copy_(first[1])
    for s in range(steps):
        x = qkv[s]
        now = (start + s + 1).to(torch.int32)
        pa.store_kv(x[:, H:H + Hkv], x[:, H + Hkv:], slots[s], kc, vc)
        torch.cuda.synchronize()
        ref = pa.decode(x[:, :H], kc, vc, bt, now, 0.1)
        torch.cuda.synchronize()
        assert torch.equal(outs[s], ref), s
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_blocks_far_into_a_large_pool(kv):
    # offsets past 2^32 elements (bf16) or bytes (E4M3): the same calls give the same bits as
    # over a pool that holds just the blocks in use
    H, Hkv, D, bs, B, width = 32, 8, 128, 16, 3, 24
    n = B * width
    g = torch.Generator().manual_seed(402)
    NB = (2 ** 32 // (Hkv * D * bs)) + 500
    lens, budget, sinks, recent = [300, 150, 384], 100, 4, 30
    T = sum(lens)
    perm = torch.randperm(n, generator=g).view(B, width).to(torch.int32)
    qkv = torch.randn((T, H + 2 * Hkv, D), generator=g).to(torch.bfloat16).cuda()
    cs = torch.from_numpy(table(512, D)).cuda()
    pos = torch.cat([torch.arange(m) for m in lens])
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(lens)])
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    got = []
    for blocks in (n, NB):
        first = blocks - n
        bt = perm + first
        slots = (bt.long()[seq, pos // bs] * bs + pos % bs).cuda()
        dt = torch.bfloat16 if kv == "bf16" else torch.uint8
        kc, vc = (torch.empty((blocks, bs, Hkv, D), dtype=dt, device="cuda") for _ in range(2))
        ks = vs = None
        if kv != "bf16":
            ks, vs = (torch.zeros((blocks, Hkv, bs), device="cuda") for _ in range(2))
        scores = torch.zeros((blocks, Hkv, bs), device="cuda")
        kc[first:] = 0
        vc[first:] = 0
        bt = bt.cuda()
        q = pa.norm_rope_store(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], pos.cuda(), slots,
                               kc, vc, cos_sin=cs, k_scale=ks, v_scale=vs, scores=scores)
        res = [q]
        if kv == "bf16":
            res.append(pa.prefill_window(q, kc, vc, bt, cu, cu, 0.1, 64, 4))
        res.append(pa.decode_scored(q[cu[1:].long() - 1], kc, vc, bt, cl, scores, 0.1, k_scale=ks,
                                    v_scale=vs))
        res += pa.evict(kc, vc, scores, bt, cl, budget, sinks=sinks, recent=recent, k_scale=ks,
                        v_scale=vs)
        res += [t[first:].clone() for t in (kc, vc, scores, ks, vs) if t is not None]
        torch.cuda.synchronize()
        assert pa.get_device_error() == 0
        got.append(res)
        del kc, vc, ks, vs, scores
        torch.cuda.empty_cache()
    for a, b in zip(*got):
        assert torch.equal(a, b)
