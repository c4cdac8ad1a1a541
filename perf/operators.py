"""The operators of a decode loop over a bounded paged KV cache, as cases to measure.

  norm_rope_store   RMS norm of every query and key head, the position rotation of both, and the
                    store of the new K and V rows in their cache slots (quantised for an 8-bit
                    cache), straight from the fused projection's output.
  prefill_window    packed varlen prefill over the paged cache where a query sees the last
                    `window` keys and the first `sinks` keys.
  decode_scored     decode attention that adds every key's softmax weight (summed over the query
                    heads of its kv head) to a score kept beside the cache.
  evict             keep `budget` keys of each sequence and kv head (the first `sinks`, the last
                    `recent`, and the best scores between them) and move them to the front.

listed() and draw() give cases, prepare() what a serving program holds before the call, run() one
call: in plain torch operations, or through the library where `own` is true. exact() is the
definition in 64 bits. Lengths follow from the case alone, values from the seed.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

FP8_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a Llama-3-8B-shaped batch: 64 tokens, latency
        dict(name="rope_store_decode_b64", op="norm_rope_store", tokens=64, kv_heads=8, group=4,
             head_dim=128, block_size=16, kv="bf16", rotary=128, interleaved=False,
             max_pos=4096, pool=20000, lens_seed=1),
        # one decode step of a continuous batch of 256 with an 8-bit cache, 64 query heads
        dict(name="rope_store_fp8_decode_b256", op="norm_rope_store", tokens=256, kv_heads=8,
             group=8, head_dim=128, block_size=32, kv="fp8", rotary=128, interleaved=False,
             max_pos=16384, pool=4000, lens_seed=2),
        # a packed prompt chunk, odd length, half of each head rotated in interleaved pairs
        dict(name="rope_store_prompt_16383", op="norm_rope_store", tokens=16383, kv_heads=8,
             group=4, head_dim=128, block_size=16, kv="bf16", rotary=64, interleaved=True,
             max_pos=131072, pool=2000, lens_seed=3),
        # short continuations (one to sixteen new tokens each) over cached prefixes
        dict(name="window_short_b32", op="prefill_window", batch=32, kv_heads=8, group=4,
             block_size=16, q_lo=1, q_hi=16, c_lo=0, c_hi=8192, window=1024, sinks=4, lens_seed=4),
        # the varlen prefix-cached prefill of the benchmark, with a window
        dict(name="window_varlen_b8", op="prefill_window", batch=8, kv_heads=8, group=4,
             block_size=16, q_lo=128, q_hi=1024, c_lo=0, c_hi=2048, window=1000, sinks=4,
             lens_seed=5),
        # two long prompts, a window of 4096
        dict(name="window_long_b2", op="prefill_window", batch=2, kv_heads=8, group=8,
             block_size=32, q_lo=9001, q_hi=16384, c_lo=0, c_hi=5000, window=4096, sinks=64,
             lens_seed=6),
        # a Llama-3-8B-shaped decode batch, contexts 512 to 4096
        dict(name="scored_b64", op="decode_scored", batch=64, kv_heads=8, group=4, head_dim=128,
             block_size=16, kv="bf16", lens="uniform", lo=512, hi=4096, lens_seed=7),
        # eight long contexts: work split over the length
        dict(name="scored_long_b8", op="decode_scored", batch=8, kv_heads=8, group=4,
             head_dim=128, block_size=16, kv="bf16", lens="uniform", lo=32768, hi=131072,
             lens_seed=8),
        # a continuous batch with an 8-bit cache, lognormal lengths
        dict(name="scored_fp8_b256", op="decode_scored", batch=256, kv_heads=8, group=8,
             head_dim=128, block_size=32, kv="fp8", lens="lognormal", lo=1, hi=16384,
             lens_seed=9),
        # a small batch that went a few steps over its budget
        dict(name="evict_b4", op="evict", batch=4, kv_heads=2, group=1, head_dim=64,
             block_size=16, kv="bf16", lens="uniform", lo=700, hi=1100, budget=512, sinks=4,
             recent=64, lens_seed=10),
        # the steady state: 64 sequences 128 tokens over a budget of 2048, 8-bit cache
        dict(name="evict_steady_fp8_b64", op="evict", batch=64, kv_heads=8, group=1,
             head_dim=128, block_size=32, kv="fp8", lens="uniform", lo=2176, hi=2176, budget=2048,
             sinks=4, recent=1024, lens_seed=11),
        # long prompts cut to a budget of 4096
        dict(name="evict_long_b8", op="evict", batch=8, kv_heads=8, group=1, head_dim=128,
             block_size=16, kv="bf16", lens="uniform", lo=32768, hi=131072, budget=4096, sinks=4,
             recent=256, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope_store", "prefill_window", "decode_scored", "evict"])
    c = dict(op=op, kv_heads=rng.choice([1, 2, 4, 8]), block_size=rng.choice([16, 32]),
             lens_seed=rng.randrange(1 << 30))
    if op == "norm_rope_store":
        c["kv"] = rng.choice(["bf16", "fp8"])
        c["head_dim"] = 128 if c["kv"] == "fp8" else rng.choice([64, 128])
        c["group"] = rng.randint(1, 8)
        c["tokens"] = _log_int(rng, 1, 16383)
        c["rotary"] = rng.choice([c["head_dim"], c["head_dim"] // 2])
        c["interleaved"] = rng.random() < 0.5
        c["max_pos"] = rng.choice([4096, 16384, 131072])
        c["pool"] = 2 * (c["tokens"] // c["block_size"] + 8)
    elif op == "prefill_window":
        c["group"] = rng.choice([1, 2, 4, 8, 16])
        c["batch"] = _log_int(rng, 1, 32)
        c["q_lo"] = 1
        c["q_hi"] = _log_int(rng, 1, max(1, 16384 // c["batch"]))
        c["c_lo"] = 0
        c["c_hi"] = _log_int(rng, 16, 8192)
        c["window"] = _log_int(rng, 1, 4096)
        c["sinks"] = rng.choice([0, 1, 4, 64])
    else:
        c["kv"] = rng.choice(["bf16", "bf16", "fp8", "int8"])
        c["head_dim"] = rng.choice([64, 128]) if c["kv"] == "bf16" else 128
        c["group"] = rng.randint(1, 8) if op == "decode_scored" else 1
        c["batch"] = _log_int(rng, 1, 256)
        c["lens"] = "uniform"
        c["hi"] = _log_int(rng, 64, min(131072, 524288 // c["batch"]))
        c["lo"] = max(1, c["hi"] // rng.choice([1, 2, 8]))
        if op == "evict":
            c["budget"] = _log_int(rng, 16, min(4096, c["hi"]))
            c["sinks"] = min(rng.choice([0, 4]), c["budget"])
            c["recent"] = rng.randint(0, c["budget"] - c["sinks"])
    return c


def _lengths(case):
    """The context lengths of a decode_scored or evict case."""
    r = random.Random(case["lens_seed"])
    if case["lens"] == "lognormal":  # median 1024, sigma 1
        return [min(case["hi"], max(case["lo"], round(1024.0 * math.exp(r.gauss(0.0, 1.0)))))
                for _ in range(case["batch"])]
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _prompt_lengths(case):
    """(cached lengths, new-token counts) of a prefill_window case."""
    r = random.Random(case["lens_seed"])
    return ([r.randint(case["c_lo"], case["c_hi"]) for _ in range(case["batch"])],
            [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])])


def _elem(case):
    return 2 if case.get("kv", "bf16") == "bf16" else 1


def work(case):
    hkv, h = case["kv_heads"], case["kv_heads"] * case["group"]
    d = case.get("head_dim", 128)
    row = d * _elem(case) + (0 if _elem(case) == 2 else 4)  # one K or V row of a head, its scale
    if case["op"] == "norm_rope_store":
        t = case["tokens"]
        return dict(bytes=t * ((2 * h + 2 * hkv) * d * 2 + 2 * hkv * row + case["rotary"] * 4 + 16),
                    flops=t * (h + hkv) * d * 8)
    if case["op"] == "prefill_window":
        w, s = case["window"], case["sinks"]
        pairs = keys = rows = 0
        for c, n in zip(*_prompt_lengths(case)):
            last = np.arange(c, c + n, dtype=np.int64)  # position of each query
            lo = np.maximum(last - w + 1, 0)
            pairs += int((last - lo + 1 + np.minimum(lo, s)).sum())
            keys += int(last[-1] + 1 - lo[0] + min(int(lo[0]), s))
            rows += n
        return dict(bytes=rows * h * d * 4 + keys * hkv * d * 4, flops=4 * d * h * pairs)
    total = sum(_lengths(case))
    if case["op"] == "decode_scored":
        return dict(bytes=total * hkv * (2 * row + 8) + case["batch"] * h * d * 4,
                    flops=4 * d * h * total)
    over = [n for n in _lengths(case) if n > case["budget"]]
    moved = len(over) * hkv * (case["budget"] - case["sinks"])
    return dict(bytes=sum(over) * hkv * 4 + moved * 2 * (2 * row + 4)
                + case["batch"] * hkv * case["budget"] * 4, flops=0)


# ------------------------------------------------------------------ inputs
def _cache(case, num_blocks, g):
    """K and V caches (num_blocks, block_size, kv_heads, head_dim) with their scales."""
    shape = (num_blocks, case["block_size"], case["kv_heads"], case.get("head_dim", 128))
    kv = case.get("kv", "bf16")
    if kv == "bf16":
        return [torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
                for _ in range(2)] + [None, None]
    caches = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if kv == "fp8":
            caches.append((x * 100.0).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
                          .view(torch.uint8))
        else:
            caches.append((x * 32.0).round_().clamp_(-127, 127).to(torch.int8))
    one = 1.0 / (100.0 if kv == "fp8" else 32.0)
    sshape = (num_blocks, case["kv_heads"], case["block_size"])
    return caches + [one * (0.5 + torch.rand(sshape, generator=g, device="cuda"))
                     for _ in range(2)]


def _tables(lens, block_size, g):
    """Physical blocks in random order: (block table int32, blocks in the pool)."""
    need = [max(1, -(-n // block_size)) for n in lens]
    pool = sum(need) + sum(need) // 16 + 1
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    first = torch.tensor(np.concatenate([[0], np.cumsum(need)[:-1]]), device="cuda")
    col = torch.arange(max(need), device="cuda")[None, :]
    real = col < torch.tensor(need, device="cuda")[:, None]
    table[real] = perm[(first[:, None] + col)[real]]
    return table, pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    hkv, h, d = case["kv_heads"], case["kv_heads"] * case["group"], case.get("head_dim", 128)
    bs = case["block_size"]
    s = dict(case=case, op=case["op"], scale=1.0 / math.sqrt(d))
    if case["op"] == "norm_rope_store":
        t = case["tokens"]
        # the fused projection's output: q, k and v are views of one tensor
        qkv = torch.randn((t, (h + 2 * hkv) * d), generator=g, device="cuda",
                          dtype=torch.bfloat16) * 3.0
        s["q"] = qkv[:, :h * d].view(t, h, d)
        s["k"] = qkv[:, h * d:(h + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (h + hkv) * d:].view(t, hkv, d)
        s["qw"], s["kw"] = (1.0 + 0.2 * torch.randn((2, d), generator=g, device="cuda")).to(
            torch.bfloat16)
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(case, case["pool"], g)
        s["slots"] = torch.randperm(case["pool"] * bs, generator=g, device="cuda")[:t].contiguous()
        if t > 8:  # padding tokens of a batch that is not full
            s["slots"][t - 2] = -1
        s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=g, device="cuda")
        half = case["rotary"] // 2
        freq = 500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        ang = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
        s["q_out"] = torch.zeros((t, h, d), dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "prefill_window":
        cached, n = _prompt_lengths(case)
        lens = [a + b for a, b in zip(cached, n)]
        s["bt"], pool = _tables(lens, bs, g)
        s["k_cache"], s["v_cache"], _, _ = _cache(case, pool, g)
        s["q"] = torch.randn((sum(n), h, d), generator=g, device="cuda", dtype=torch.bfloat16) * 2.0
        s["cu_q"], s["cu_k"] = (torch.tensor(np.concatenate([[0], np.cumsum(x)]),
                                             dtype=torch.int32, device="cuda") for x in (n, lens))
        s["n"], s["lens"], s["max_q"] = n, lens, max(n)
        s["out"] = torch.empty_like(s["q"])
        return s
    lens = _lengths(case)
    s["bt"], pool = _tables(lens, bs, g)
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(case, pool, g)
    s["lens"], s["max_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens)
    # accumulated weights: heavy-tailed, some keys with none at all
    sc = torch.randn((pool, hkv, bs), generator=g, device="cuda").mul_(2.0).exp_()
    s["scores"] = sc.mul_(torch.rand(sc.shape, generator=g, device="cuda") > 0.05)
    if case["op"] == "decode_scored":
        s["q"] = torch.randn((len(lens), h, d), generator=g, device="cuda",
                             dtype=torch.bfloat16) * 2.0
        s["out"] = torch.empty_like(s["q"])
    else:
        s["kept"] = torch.empty((len(lens), hkv, case["budget"]), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty_like(s["lens"])
    return s


# ------------------------------------------------------------------ plain forms
def _values(cache, scale, slots):
    """Rows of a cache in fp32: (..., kv_heads, head_dim) for slots (...)."""
    nb, bs, hkv, d = cache.shape
    x = cache.view(nb * bs, hkv, d)[slots]
    if scale is None:
        return x.float()
    if cache.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn)
    return x.float() * scale.permute(0, 2, 1).reshape(nb * bs, hkv)[slots][..., None]


def _slots(bt, block_size, n):
    """Slot of positions 0..n-1 of every sequence (0 where the table has no block)."""
    p = torch.arange(n, device=bt.device)
    return bt[:, p // block_size].clamp_min(0).long() * block_size + p % block_size


def _rotate(x, cs, interleaved):
    r = cs.shape[-1]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y, x[..., r:]], dim=-1)


def _plain_norm_rope_store(s):
    cs = s["cos_sin"][s["positions"]]
    real = s["slots"] >= 0

    def norm(x, w):
        x = x.float()
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()

    q = _rotate(norm(s["q"], s["qw"]), cs, s["case"]["interleaved"]).to(torch.bfloat16)
    s["q_out"][real] = q[real]
    k = _rotate(norm(s["k"], s["kw"]), cs, s["case"]["interleaved"])
    slots = s["slots"][real]
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (s["v"].float(), s["v_cache"],
                                                              s["v_scale"])):
        nb, bs, hkv, d = cache.shape
        x = x[real]
        if scale is not None:
            amax = x.abs().amax(-1)
            one = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
            scale[slots // bs, :, slots % bs] = one
            x = (x / one[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
            cache.view(nb * bs, hkv, d)[slots] = x.view(torch.uint8)
        else:
            cache.view(nb * bs, hkv, d)[slots] = x.to(torch.bfloat16)


def _plain_prefill_window(s):
    w, sinks, bs = s["case"]["window"], s["case"]["sinks"], s["case"]["block_size"]
    h, d = s["q"].shape[1:]
    hkv = s["case"]["kv_heads"]
    row0 = 0
    for b, (n, total) in enumerate(zip(s["n"], s["lens"])):
        slots = _slots(s["bt"][b:b + 1], bs, total)[0]
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            p = torch.arange(total - n + i0, total - n + i1, device="cuda")
            lo = max(0, total - n + i0 - w + 1)
            j = torch.cat([torch.arange(min(sinks, lo), device="cuda"),
                           torch.arange(lo, total - n + i1, device="cuda")])
            k = _values(s["k_cache"], None, slots[j]).permute(1, 2, 0)
            v = _values(s["v_cache"], None, slots[j]).permute(1, 0, 2)
            q = s["q"][row0 + i0:row0 + i1].float().view(i1 - i0, hkv, h // hkv, d)
            x = torch.matmul(q.permute(1, 2, 0, 3).reshape(hkv, -1, d), k) * s["scale"]
            x = x.view(hkv, h // hkv, i1 - i0, -1)
            seen = (j <= p[:, None]) & ((j < sinks) | (j > p[:, None] - w))
            x = x.masked_fill_(~seen, -math.inf)
            x = (x - x.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(x.view(hkv, -1, x.shape[-1]), v).view(hkv, h // hkv, i1 - i0, d)
            o = o / x.sum(-1, keepdim=True)
            s["out"][row0 + i0:row0 + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, h, d).to(
                torch.bfloat16)
        row0 += n


def _plain_decode_scored(s):
    b, h, d = s["q"].shape
    nb, bs, hkv, _ = s["k_cache"].shape
    n = s["max_len"]
    slots = _slots(s["bt"], bs, n)
    real = torch.arange(n, device="cuda") < s["lens"][:, None]
    k = _values(s["k_cache"], s["k_scale"], slots).permute(0, 2, 3, 1)
    x = torch.matmul(s["q"].float().view(b, hkv, h // hkv, d), k) * s["scale"]
    del k
    x = x.masked_fill_(~real[:, None, None, :], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp_()
    x = x / x.sum(-1, keepdim=True)
    v = _values(s["v_cache"], s["v_scale"], slots).permute(0, 2, 1, 3)
    s["out"].copy_(torch.matmul(x, v).view(b, h, d))
    at = (slots // bs * hkv * bs + slots % bs)[:, :, None] + torch.arange(hkv, device="cuda") * bs
    s["scores"].view(-1).index_add_(0, at[real].view(-1),
                                    x.sum(2).permute(0, 2, 1)[real].reshape(-1))


def _plain_evict(s):
    c = s["case"]
    budget, n, bs = c["budget"], s["max_len"], c["block_size"]
    nb, _, hkv, d = s["k_cache"].shape
    lens, p = s["lens"].long(), torch.arange(max(s["max_len"], budget), device="cuda")
    slots = _slots(s["bt"], bs, n)
    x = s["scores"].permute(0, 2, 1).reshape(nb * bs, hkv)[slots].permute(0, 2, 1)
    x = torch.nn.functional.pad(x, (0, len(p) - n))
    # the first, the last and (for a sequence within its budget) all keys come before the others,
    # what is past the end after them; equal scores in the order of their positions
    always = (p < c["sinks"]) | (p >= (lens - c["recent"])[:, None]) | (lens <= budget)[:, None]
    x = x.masked_fill(always[:, None, :], math.inf)
    x = x.masked_fill((p >= lens[:, None])[:, None, :], -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :budget]
    new = lens.clamp_max(budget)
    real = (p[:budget] < new[:, None])[:, None, :].expand(-1, hkv, -1)
    order = order.masked_fill(~real, n + budget).sort(-1).values.masked_fill_(~real, -1)
    s["kept"].copy_(order)
    s["new_lens"].copy_(new)
    # rows i of (sequence, head) come from row kept[i]
    real = real & (lens > budget)[:, None, None]
    seq, head, to = real.nonzero(as_tuple=True)
    src, dst = slots[seq, order[real]], slots[seq, to]
    for t in (s["k_cache"], s["v_cache"]):
        rows = t.view(nb * bs, hkv, d)
        rows[dst, head] = rows[src, head]
    for t in (s["scores"], s["k_scale"], s["v_scale"]):
        if t is not None:
            t[dst // bs, head, dst % bs] = t[src // bs, head, src % bs]


def _state(cache):
    """A cache as a tensor of the values its codes stand for (before the scale)."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_186_gb300 as pa
        c = s["case"]
        if op == "norm_rope_store":
            pa.norm_rope_store(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"],
                               s["v_cache"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                               cos_sin=s["cos_sin"], interleaved=c["interleaved"],
                               q_out=s["q_out"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        elif op == "prefill_window":
            pa.prefill_window(s["q"], s["k_cache"], s["v_cache"], s["bt"], s["cu_q"], s["cu_k"],
                              s["scale"], c["window"], c["sinks"], max_q_len=s["max_q"],
                              out=s["out"])
        elif op == "decode_scored":
            if "workspace" not in s:  # kept for the program's life, as for decode
                b, h, _ = s["q"].shape
                s["workspace"] = torch.empty(pa.decode_scored_workspace_size(
                    s["k_cache"], b, h, s["bt"].shape[1], s["max_len"], k_scale=s["k_scale"],
                    v_scale=s["v_scale"]), dtype=torch.uint8, device="cuda")
            pa.decode_scored(s["q"], s["k_cache"], s["v_cache"], s["bt"], s["lens"], s["scores"],
                             s["scale"], max_context_len=s["max_len"], out=s["out"],
                             workspace=s["workspace"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"])
        else:
            pa.evict(s["k_cache"], s["v_cache"], s["scores"], s["bt"], s["lens"], c["budget"],
                     sinks=c["sinks"], recent=c["recent"], max_context_len=s["max_len"],
                     kept=s["kept"], new_lens=s["new_lens"], k_scale=s["k_scale"],
                     v_scale=s["v_scale"])
    elif op == "norm_rope_store":
        _plain_norm_rope_store(s)
    elif op == "prefill_window":
        _plain_prefill_window(s)
    elif op == "decode_scored":
        _plain_decode_scored(s)
    else:
        _plain_evict(s)
    if op == "norm_rope_store":
        return [s["q_out"], _state(s["k_cache"]), _state(s["v_cache"]), s["k_scale"], s["v_scale"]]
    if op == "prefill_window":
        return [s["out"]]
    if op == "decode_scored":
        return [s["out"], s["scores"]]
    return [s["kept"], s["new_lens"], _state(s["k_cache"]), _state(s["v_cache"]), s["scores"],
            s["k_scale"], s["v_scale"]]


# ------------------------------------------------------------------ definitions in 64 bits
def _rows64(cache, scale, phys, off):
    """Rows (block phys, offset off) of a cache in 64 bits: (n, kv_heads, head_dim)."""
    x = cache[phys, off] if cache.dtype != torch.uint8 else cache[phys, off].view(
        torch.float8_e4m3fn)
    x = x.double()
    return x if scale is None else x * scale[phys, :, off].double()[:, :, None]


def _exact_norm_rope_store(s):
    c = s["case"]
    d, r, bs = c["head_dim"], c["rotary"], c["block_size"]
    first = list(range(0, r, 2)) if c["interleaved"] else list(range(r // 2))
    second = [i + 1 for i in first] if c["interleaved"] else [i + r // 2 for i in first]
    ang = s["cos_sin"][s["positions"]].double()
    cos, sin = ang[:, None, :r // 2], ang[:, None, r // 2:]

    def turned(x, w):
        x = x.double()
        x = x * w.double() / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d
                                        + 1e-6)
        y = x.clone()
        y[..., first] = x[..., first] * cos - x[..., second] * sin
        y[..., second] = x[..., second] * cos + x[..., first] * sin
        return y

    q, k, v = turned(s["q"], s["qw"]), turned(s["k"], s["kw"]), s["v"].double()
    live = torch.nonzero(s["slots"] >= 0).flatten()
    phys, off = s["slots"][live] // bs, s["slots"][live] % bs
    out_q = s["q_out"].double()
    out_q[live] = q[live]
    if c["kv"] == "bf16":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc[phys, off], vc[phys, off] = k[live], v[live]
        return [out_q, kc, vc, None, None]
    scales = [s["k_scale"].double(), s["v_scale"].double()]
    caches = [s["k_cache"].view(torch.float8_e4m3fn).double(),
              s["v_cache"].view(torch.float8_e4m3fn).double()]
    for x, cache, scale in zip((k, v), caches, scales):
        top = x[live].abs().max(dim=-1).values / FP8_MAX
        top[top == 0] = 1.0
        scale[phys, :, off] = top
        cache[phys, off] = x[live] / top[..., None]  # before the rounding to the code
    return [out_q, caches[0], caches[1], scales[0], scales[1]]


def _exact_prefill_window(s):
    c = s["case"]
    w, sinks, bs, hkv, grp = c["window"], c["sinks"], c["block_size"], c["kv_heads"], c["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    r0 = 0
    for b in range(c["batch"]):
        n, total = s["n"][b], s["lens"][b]
        j = torch.arange(total, device="cuda")
        phys, off = s["bt"][b][j // bs].long(), j % bs
        for at in range(0, n, 512):
            i = torch.arange(at, min(n, at + 512), device="cuda")
            last = int(i[-1]) + total - n
            start = max(0, int(i[0]) + total - n - w + 1)
            cols = torch.nonzero((j <= last) & ((j >= start) | (j < sinks))).flatten()
            k = _rows64(s["k_cache"], None, phys[cols], off[cols])
            v = _rows64(s["v_cache"], None, phys[cols], off[cols])
            age = (i + total - n)[:, None] - cols[None, :]
            bias = torch.zeros(age.shape, dtype=torch.float64, device="cuda")
            bias[(age < 0) | ((age >= w) & (cols >= sinks)[None, :])] = -math.inf
            q = s["q"][r0 + i].double()
            for head in range(hkv):
                for m in range(grp):
                    logit = (q[:, head * grp + m] @ k[:, head].T) * s["scale"] + bias
                    weight = torch.exp(logit - torch.logsumexp(logit, dim=1, keepdim=True))
                    out[r0 + i, head * grp + m] = weight @ v[:, head]
        r0 += n
    return [out]


def _exact_decode_scored(s):
    c = s["case"]
    bs, hkv, grp = c["block_size"], c["kv_heads"], c["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    scores = s["scores"].double()
    for b, n in enumerate(s["lens"].tolist()):
        j = torch.arange(n, device="cuda")
        phys, off = s["bt"][b][j // bs].long(), j % bs
        k = _rows64(s["k_cache"], s["k_scale"], phys, off)
        v = _rows64(s["v_cache"], s["v_scale"], phys, off)
        q = s["q"][b].double().view(hkv, grp, -1)
        logit = torch.einsum("hgd,nhd->hgn", q, k) * s["scale"]
        weight = torch.exp(logit - torch.logsumexp(logit, dim=2, keepdim=True))
        out[b] = torch.einsum("hgn,nhd->hgd", weight, v).reshape(hkv * grp, -1)
        scores[phys, :, off] += weight.sum(1).T
    return [out, scores]


def _exact_evict(s):
    c = s["case"]
    bs, hkv, budget = c["block_size"], c["kv_heads"], c["budget"]
    kept = np.full((c["batch"], hkv, budget), -1, dtype=np.int32)
    tables, lens = s["bt"].cpu().numpy(), s["lens"].cpu().numpy()
    scores = s["scores"].cpu().numpy()
    dst, src = [], []
    for b, n in enumerate(lens.tolist()):
        j = np.arange(n)
        phys, off = tables[b][j // bs].astype(np.int64), j % bs
        for head in range(hkv):
            if n <= budget:
                kept[b, head, :n] = j
                continue
            mid = np.arange(c["sinks"], n - c["recent"])
            val = scores[phys[mid], head, off[mid]]
            best = mid[np.lexsort((mid, -val))[:budget - c["sinks"] - c["recent"]]]
            keep = np.sort(np.concatenate([np.arange(c["sinks"]), best,
                                           np.arange(n - c["recent"], n)]))
            kept[b, head] = keep
            one = np.full(budget, head)
            src.append(np.stack([phys[keep], off[keep], one]))
            dst.append(np.stack([phys[:budget], off[:budget], one]))
    got = [torch.from_numpy(kept), torch.from_numpy(np.minimum(lens, budget).astype(np.int32))]
    a = b = None
    if dst:
        a, b = (torch.from_numpy(np.concatenate(x, axis=1)).cuda() for x in (dst, src))
    for t, by_slot in ((_state(s["k_cache"]), True), (_state(s["v_cache"]), True),
                       (s["scores"], False), (s["k_scale"], False), (s["v_scale"], False)):
        if t is not None and a is not None:
            raw = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
            new = raw.clone()
            if by_slot:
                new[a[0], a[1], a[2]] = raw[b[0], b[1], b[2]]
            else:
                new[a[0], a[2], a[1]] = raw[b[0], b[2], b[1]]
            t = new.view(t.dtype)
        got.append(t)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope_store": _exact_norm_rope_store, "prefill_window": _exact_prefill_window,
            "decode_scored": _exact_decode_scored, "evict": _exact_evict}[case["op"]](s)
