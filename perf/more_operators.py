"""The operators of serving many requests over one shared context, as cases to measure.

A batch often shares a long beginning: many questions about one document or video, many samples
of one prompt, a few system prompts in front of every request. Its blocks are in the cache once
and every sequence's block table begins with them.

  norm_rope_axes_store  RMS norm of every query and key head, the rotation of each pair of dims by
                        the position on that pair's own axis (time, height, width), and the store
                        of the new K and V rows in their cache slots.
  decode_shared         decode attention of groups of sequences whose block tables begin with the
                        same blocks: the shared keys are attended to once for a whole group.
  prefill_shared        packed varlen prefill of the new tokens of such sequences (questions over
                        one document, drafts to verify).

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
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 conversations about images: the new tokens' three positions agree
        # no more with their place in the sequence, latency
        dict(name="axes_decode_b64", op="norm_rope_axes_store", tokens=64, kv_heads=8, group=4,
             head_dim=128, block_size=16, kv="bf16", rotary=128, interleaved=False,
             layout="sections", axes=3, max_pos=4096, pool=20000),
        # images in a prompt, 8-bit cache, pairs dealt out to height and width in turn
        dict(name="axes_image_fp8_4097", op="norm_rope_axes_store", tokens=4097, kv_heads=8,
             group=8, head_dim=128, block_size=32, kv="fp8", rotary=128, interleaved=True,
             layout="cycle", axes=2, max_pos=1024, pool=1000),
        # a video in a prompt: time, height and width in sections of the rotated half
        dict(name="axes_video_16383", op="norm_rope_axes_store", tokens=16383, kv_heads=8, group=4,
             head_dim=128, block_size=16, kv="bf16", rotary=128, interleaved=False,
             layout="sections", axes=3, max_pos=16384, pool=2000),
        # four samples of one short prompt: latency
        dict(name="shared_b4", op="decode_shared", batch=4, groups=1, kv_heads=8, group=4,
             head_dim=128, block_size=16, kv="bf16", p_lo=1000, p_hi=1000, o_lo=1, o_hi=64, pad=0,
             lens_seed=1),
        # 64 samples of one prompt, an odd prefix length
        dict(name="shared_b64", op="decode_shared", batch=64, groups=1, kv_heads=8, group=4,
             head_dim=128, block_size=16, kv="bf16", p_lo=8191, p_hi=8191, o_lo=1, o_hi=512, pad=0,
             lens_seed=2),
        # a continuous batch behind sixteen system prompts, not full: the last rows are padding
        dict(name="shared_groups_b128", op="decode_shared", batch=128, groups=16, kv_heads=8,
             group=4, head_dim=64, block_size=16, kv="bf16", p_lo=500, p_hi=8000, o_lo=1,
             o_hi=1000, pad=5, lens_seed=3),
        # 256 requests over one long prompt, 64 query heads, 8-bit cache
        dict(name="shared_fp8_b256", op="decode_shared", batch=256, groups=1, kv_heads=8, group=8,
             head_dim=128, block_size=32, kv="fp8", p_lo=16384, p_hi=16384, o_lo=1, o_hi=1024,
             pad=0, lens_seed=4),
        # 32 questions being answered over one long document: bound by reading it
        dict(name="shared_document_b32", op="decode_shared", batch=32, groups=1, kv_heads=8,
             group=4, head_dim=128, block_size=16, kv="bf16", p_lo=131067, p_hi=131067, o_lo=1,
             o_hi=256, pad=0, lens_seed=5),
        # drafts of four to eight tokens to verify, 64 requests behind one prompt
        dict(name="drafts_b64", op="prefill_shared", batch=64, groups=1, kv_heads=8, group=4,
             block_size=16, p_lo=4096, p_hi=4096, o_lo=0, o_hi=512, q_lo=4, q_hi=8, lens_seed=6),
        # 32 questions of up to 64 tokens over one document
        dict(name="questions_b32", op="prefill_shared", batch=32, groups=1, kv_heads=8, group=4,
             block_size=16, p_lo=8000, p_hi=8000, o_lo=0, o_hi=0, q_lo=1, q_hi=64, lens_seed=7),
        # four long documents, sixteen questions of up to 256 tokens each
        dict(name="questions_groups_b64", op="prefill_shared", batch=64, groups=4, kv_heads=8,
             group=4, block_size=32, p_lo=8192, p_hi=16384, o_lo=0, o_hi=100, q_lo=16, q_hi=256,
             lens_seed=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope_axes_store", "decode_shared", "decode_shared", "prefill_shared"])
    c = dict(op=op, kv_heads=rng.choice([1, 2, 4, 8]), block_size=rng.choice([16, 32]))
    if op == "norm_rope_axes_store":
        c["kv"] = rng.choice(["bf16", "fp8"])
        c["head_dim"] = rng.choice([64, 128]) if c["kv"] == "bf16" else 128
        c["group"] = rng.randint(1, 8)
        c["tokens"] = _log_int(rng, 1, 16383)
        c["rotary"] = rng.choice([c["head_dim"], c["head_dim"] // 2])
        c["interleaved"] = rng.random() < 0.5
        c["layout"] = rng.choice(["sections", "cycle"])
        c["axes"] = rng.randint(1, 4)
        c["max_pos"] = rng.choice([1024, 4096, 16384])
        c["pool"] = 2 * (c["tokens"] // c["block_size"] + 8)
        return c
    c["lens_seed"] = rng.randrange(1 << 30)
    if op == "decode_shared":
        c["kv"] = rng.choice(["bf16", "bf16", "fp8", "int8"])
        c["head_dim"] = rng.choice([64, 128]) if c["kv"] == "bf16" else 128
        c["group"] = rng.randint(1, 8)
        c["batch"] = _log_int(rng, 1, 256)
        c["groups"] = rng.randint(1, min(c["batch"], 16))
        c["p_hi"] = _log_int(rng, 16, min(131072, 4194304 // c["batch"], 114688 // c["groups"]))
        c["p_lo"] = max(1, c["p_hi"] // rng.choice([1, 2, 8]))
        c["o_lo"] = 1
        c["o_hi"] = _log_int(rng, 1, min(4096, 131072 // c["batch"]))
        c["pad"] = rng.choice([0, 0, 1, 3]) if c["batch"] > 8 else 0
    else:
        c["group"] = rng.choice([1, 2, 4, 8, 16])
        c["batch"] = _log_int(rng, 1, 64)
        c["groups"] = rng.randint(1, min(c["batch"], 8))
        c["q_lo"] = 1
        c["q_hi"] = _log_int(rng, 1, max(1, 4096 // c["batch"]))
        c["p_hi"] = _log_int(rng, 16, min(16384, 114688 // c["groups"]))
        c["p_lo"] = max(1, c["p_hi"] // rng.choice([1, 2, 8]))
        c["o_lo"] = 0
        c["o_hi"] = rng.choice([0, 1, 100, 1000])
    return c


def _plan(case):
    """Lengths of an attention case: group bounds, prefix per group, (own cached, new) per
    sequence. A decode step's new token is its one query; a padding row has no keys."""
    r = random.Random(case["lens_seed"])
    n, groups = case["batch"], case["groups"]
    cu = [0] + sorted(r.sample(range(1, n), groups - 1)) + [n]
    prefix = [r.randint(case["p_lo"], case["p_hi"]) for _ in range(groups)]
    if case["op"] == "decode_shared":
        rows = [(r.randint(case["o_lo"], case["o_hi"]) - 1, 1) for _ in range(n)]
    else:
        rows = [(r.randint(case["o_lo"], case["o_hi"]), r.randint(case["q_lo"], case["q_hi"]))
                for _ in range(n)]
    group_of = [g for g in range(groups) for _ in range(cu[g], cu[g + 1])]
    lens = [prefix[group_of[b]] + o + q for b, (o, q) in enumerate(rows)]
    for b in range(n - case.get("pad", 0), n):
        lens[b] = 0
    return cu, prefix, group_of, [q for _, q in rows], lens


def _elem(case):
    return 2 if case.get("kv", "bf16") == "bf16" else 1


def work(case):
    hkv, h = case["kv_heads"], case["kv_heads"] * case["group"]
    d = case.get("head_dim", 128)
    row = d * _elem(case) + (0 if _elem(case) == 2 else 4)  # one K or V row of a head, its scale
    if case["op"] == "norm_rope_axes_store":
        t = case["tokens"]
        return dict(bytes=t * ((2 * h + 2 * hkv) * d * 2 + 2 * hkv * row + case["rotary"] * 4
                               + case["axes"] * 8 + 8), flops=t * (h + hkv) * d * 8)
    cu, prefix, group_of, new, lens = _plan(case)
    keys = pairs = rows = 0
    for g, p in enumerate(prefix):
        if any(lens[cu[g]:cu[g + 1]]):
            keys += p
    for b, n in enumerate(lens):
        rows += new[b]
        if n:
            keys += n - prefix[group_of[b]]
            pairs += new[b] * n - new[b] * (new[b] - 1) // 2
    return dict(bytes=keys * hkv * 2 * row + rows * h * d * 4, flops=4 * d * h * pairs)


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


def _pair_axis(case):
    """The axis of every rotated pair: contiguous sections, the first about half as long as the
    others (time), or dealt out in turn."""
    half, axes = case["rotary"] // 2, case["axes"]
    if case["layout"] == "cycle" or axes == 1:
        return [i % axes for i in range(half)]
    first = half // (2 * axes - 1)
    return [0 if i < first else 1 + (i - first) * (axes - 1) // (half - first)
            for i in range(half)]


def _positions(case, g):
    """(axes, tokens): text, whose axes agree, with grids of an image or a video's frames in it."""
    t, axes, top = case["tokens"], case["axes"], case["max_pos"]
    at = torch.arange(t, device="cuda")
    kinds = [at // 1024, at // 32 % 32, at % 32, at % 7]  # frame, row, column, one more
    grid = torch.stack(kinds[1:3] if axes == 2 else kinds[:axes])
    start = torch.randint(0, max(1, top - 1 - int(grid.max())), (t // 4096 + 1,), generator=g,
                          device="cuda")
    text = torch.rand((t // 64 + 1,), generator=g, device="cuda")[at // 64] < 0.25
    base = start[at // 4096][None, :]
    pos = torch.where(text[None, :], base + (at % 32)[None, :], base + grid)
    return pos.clamp_(0, top - 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    hkv, h, d = case["kv_heads"], case["kv_heads"] * case["group"], case.get("head_dim", 128)
    bs = case["block_size"]
    s = dict(case=case, op=case["op"], scale=1.0 / math.sqrt(d))
    if case["op"] == "norm_rope_axes_store":
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
        s["positions"] = _positions(case, g)
        s["pair_axis"] = _pair_axis(case)
        s["axis"] = torch.tensor(s["pair_axis"], device="cuda")
        half = case["rotary"] // 2
        freq = 500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        ang = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
        s["q_out"] = torch.zeros((t, h, d), dtype=torch.bfloat16, device="cuda")
        return s
    cu, prefix, group_of, new, lens = _plan(case)
    # physical blocks in random order: a group's shared blocks once, then each sequence's own
    shared = [p // bs for p in prefix]
    mine = [max(0, -(-n // bs) - shared[group_of[b]]) for b, n in enumerate(lens)]
    width = max(max(shared), max(m + shared[group_of[b]] for b, m in enumerate(mine)), 1)
    pool = sum(shared) + sum(mine) + (sum(shared) + sum(mine)) // 16 + 1
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table = np.full((len(lens), width), -1, dtype=np.int32)
    heads, at = [], 0
    for n in shared:
        heads.append(perm[at:at + n])
        at += n
    for b, m in enumerate(mine):
        if lens[b]:
            n = shared[group_of[b]]
            table[b, :n] = heads[group_of[b]]
            table[b, n:n + m] = perm[at:at + m]
            at += m
    s["bt"] = torch.from_numpy(table).cuda()
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(case, pool, g)
    s["cu_groups"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    # what the host knows of the lengths, as a scheduler does
    s["cu"], s["prefix"], s["new"], s["host_lens"] = cu, prefix, new, lens
    s["max_len"] = max(max(lens), 1)
    s["q"] = torch.randn((sum(new), h, d), generator=g, device="cuda", dtype=torch.bfloat16) * 2.0
    s["out"] = torch.empty_like(s["q"])
    if case["op"] == "decode_shared":
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    else:
        s["cu_q"], s["cu_k"] = (torch.tensor(np.concatenate([[0], np.cumsum(x)]),
                                             dtype=torch.int32, device="cuda") for x in (new, lens))
        s["max_q"] = max(new)
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


def _slots(bt, block_size, first, last):
    """Slots of positions first..last-1 of every row of a block table (0 where it has no block)."""
    p = torch.arange(first, last, device=bt.device)
    j = (p // block_size).clamp_max(bt.shape[1] - 1)
    return bt[:, j].clamp_min(0).long() * block_size + p % block_size


def _plain_norm_rope_axes_store(s):
    inter, r = s["case"]["interleaved"], s["case"]["rotary"]
    half = r // 2
    pair = torch.arange(half, device="cuda")
    at = s["positions"][s["axis"]].T  # (tokens, pairs): every pair's own position
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, half + pair][:, None]
    real = s["slots"] >= 0

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :half], x[..., half:r])
        y = [a * cos - b * sin, b * cos + a * sin]
        y = torch.stack(y, dim=-1).flatten(-2) if inter else torch.cat(y, dim=-1)
        return torch.cat([y, x[..., r:]], dim=-1)

    s["q_out"][real] = turned(s["q"], s["qw"]).to(torch.bfloat16)[real]
    slots = s["slots"][real]
    for x, cache, scale in ((turned(s["k"], s["kw"]), s["k_cache"], s["k_scale"]),
                            (s["v"].float(), s["v_cache"], s["v_scale"])):
        nb, bs, hkv, d = cache.shape
        x = x[real]
        if scale is None:
            cache.view(nb * bs, hkv, d)[slots] = x.to(torch.bfloat16)
            continue
        amax = x.abs().amax(-1)
        one = torch.where(amax > 0, amax / FP8_MAX, torch.ones_like(amax))
        scale[slots // bs, :, slots % bs] = one
        x = (x / one[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        cache.view(nb * bs, hkv, d)[slots] = x.view(torch.uint8)


def _plain_decode_shared(s):
    b, h, d = s["q"].shape
    nb, bs, hkv, _ = s["k_cache"].shape
    for g, p in enumerate(s["prefix"]):
        i0, i1 = s["cu"][g], s["cu"][g + 1]
        n, p = i1 - i0, p // bs * bs
        lens, bt = s["lens"][i0:i1], s["bt"][i0:i1]
        end = max(s["host_lens"][i0:i1])
        if end == 0:  # padding rows only
            s["out"][i0:i1] = 0
            continue
        q = s["q"][i0:i1].float().view(n, hkv, h // hkv, d)
        owner = s["host_lens"].index(end, i0, i1)
        sh = _slots(s["bt"][owner:owner + 1], bs, 0, min(p, end))[0]  # the group's, read once
        mine = _slots(bt, bs, min(p, end), end)
        k = _values(s["k_cache"], s["k_scale"], sh).permute(1, 2, 0)
        qs = q.permute(1, 0, 2, 3).reshape(hkv, n * (h // hkv), d)
        xs = torch.matmul(qs, k).view(hkv, n, h // hkv, -1).permute(1, 0, 2, 3) * s["scale"]
        del k
        k = _values(s["k_cache"], s["k_scale"], mine).permute(0, 2, 3, 1)
        xm = torch.matmul(q, k) * s["scale"]
        del k
        x = torch.cat([xs, xm], dim=-1)
        real = torch.arange(x.shape[-1], device="cuda") < lens[:, None]
        x = x.masked_fill_(~real[:, None, None, :], -math.inf)
        x = (x - x.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
        x = x / x.sum(-1, keepdim=True).clamp_min(1e-30)
        v = _values(s["v_cache"], s["v_scale"], sh).permute(1, 0, 2)
        ps = x[..., :len(sh)].permute(1, 0, 2, 3).reshape(hkv, n * (h // hkv), -1)
        o = torch.matmul(ps, v).view(hkv, n, h // hkv, d).permute(1, 0, 2, 3)
        v = _values(s["v_cache"], s["v_scale"], mine).permute(0, 2, 1, 3)
        o = o + torch.matmul(x[..., len(sh):], v)
        s["out"][i0:i1] = o.reshape(n, h, d).to(torch.bfloat16)


def _plain_prefill_shared(s):
    bs, hkv = s["case"]["block_size"], s["case"]["kv_heads"]
    h, d = s["q"].shape[1:]
    row = 0
    for g, p in enumerate(s["prefix"]):
        p = p // bs * bs
        sh = _slots(s["bt"][s["cu"][g]:s["cu"][g] + 1], bs, 0, p)[0]
        ks = _values(s["k_cache"], None, sh).permute(1, 2, 0)
        vs = _values(s["v_cache"], None, sh).permute(1, 0, 2)
        for b in range(s["cu"][g], s["cu"][g + 1]):
            n, total = s["new"][b], s["host_lens"][b]
            slots = _slots(s["bt"][b:b + 1], bs, p, total)[0]
            k = torch.cat([ks, _values(s["k_cache"], None, slots).permute(1, 2, 0)], dim=-1)
            v = torch.cat([vs, _values(s["v_cache"], None, slots).permute(1, 0, 2)], dim=1)
            at = torch.arange(total - n, total, device="cuda")
            q = s["q"][row:row + n].float().view(n, hkv, h // hkv, d)
            x = torch.matmul(q.permute(1, 2, 0, 3).reshape(hkv, -1, d), k) * s["scale"]
            x = x.view(hkv, h // hkv, n, total)
            x = x.masked_fill_(torch.arange(total, device="cuda") > at[:, None], -math.inf)
            x = (x - x.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(x.view(hkv, -1, total), v).view(hkv, h // hkv, n, d)
            o = o / x.sum(-1, keepdim=True)
            s["out"][row:row + n] = o.permute(2, 0, 1, 3).reshape(n, h, d).to(torch.bfloat16)
            row += n


def _state(cache):
    """A cache as a tensor of the values its codes stand for (before the scale)."""
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def run(s):
    op, c = s["op"], s["case"]
    if own:
        import paged_kv_cache_186_gb300 as pa
        if op == "norm_rope_axes_store":
            pa.norm_rope_axes_store(
                s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                s["pair_axis"], s["cos_sin"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                interleaved=c["interleaved"], q_out=s["q_out"], k_scale=s["k_scale"],
                v_scale=s["v_scale"])
        elif op == "decode_shared":
            if "workspace" not in s:  # kept for the program's life, as for decode
                b, h, _ = s["q"].shape
                s["workspace"] = torch.empty(pa.decode_shared_workspace_size(
                    s["k_cache"], b, h, s["bt"].shape[1], c["groups"], s["max_len"],
                    k_scale=s["k_scale"], v_scale=s["v_scale"]), dtype=torch.uint8, device="cuda")
            pa.decode_shared(s["q"], s["k_cache"], s["v_cache"], s["bt"], s["lens"],
                             s["cu_groups"], s["prefix_lens"], s["scale"],
                             max_context_len=s["max_len"], out=s["out"], workspace=s["workspace"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"])
        else:
            if "workspace" not in s:
                t, h, _ = s["q"].shape
                s["workspace"] = torch.empty(pa.prefill_shared_workspace_size(
                    s["k_cache"], t, h, c["groups"]), dtype=torch.uint8, device="cuda")
            pa.prefill_shared(s["q"], s["k_cache"], s["v_cache"], s["bt"], s["cu_q"], s["cu_k"],
                              s["cu_groups"], s["prefix_lens"], s["scale"], max_q_len=s["max_q"],
                              out=s["out"], workspace=s["workspace"])
    elif op == "norm_rope_axes_store":
        _plain_norm_rope_axes_store(s)
    elif op == "decode_shared":
        _plain_decode_shared(s)
    else:
        _plain_prefill_shared(s)
    if op == "norm_rope_axes_store":
        return [s["q_out"], _state(s["k_cache"]), _state(s["v_cache"]), s["k_scale"], s["v_scale"]]
    return [s["out"]]


# ------------------------------------------------------------------ definitions in 64 bits
def _rows64(cache, scale, phys, off):
    """Rows (block phys, offset off) of a cache in 64 bits: (n, kv_heads, head_dim)."""
    x = cache[phys, off] if cache.dtype != torch.uint8 else cache[phys, off].view(
        torch.float8_e4m3fn)
    x = x.double()
    return x if scale is None else x * scale[phys, :, off].double()[:, :, None]


def _exact_norm_rope_axes_store(s):
    c = s["case"]
    d, r, bs = c["head_dim"], c["rotary"], c["block_size"]
    cols = [s["cos_sin"][s["positions"][a]].double() for a in range(c["axes"])]

    def turned(x, w):
        x = x.double()
        x = x * w.double() / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d
                                        + EPS)
        y = x.clone()
        for i, axis in enumerate(s["pair_axis"]):
            j, k = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
            co, si = cols[axis][:, i:i + 1], cols[axis][:, r // 2 + i:r // 2 + i + 1]
            y[..., j] = x[..., j] * co - x[..., k] * si
            y[..., k] = x[..., k] * co + x[..., j] * si
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
    caches = [_state(t).double() for t in (s["k_cache"], s["v_cache"])]
    for x, cache, scale in zip((k, v), caches, scales):
        top = x[live].abs().max(dim=-1).values / FP8_MAX
        top[top == 0] = 1.0
        scale[phys, :, off] = top
        cache[phys, off] = x[live] / top[..., None]  # before the rounding to the code
    return [out_q] + caches + scales


def _exact_attention(s):
    c = s["case"]
    bs, hkv, grp = c["block_size"], c["kv_heads"], c["group"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    r0 = 0
    for b, total in enumerate(s["host_lens"]):
        n = s["new"][b]
        if total:
            j = torch.arange(total, device="cuda")
            phys, off = s["bt"][b][j // bs].long(), j % bs
            k = _rows64(s["k_cache"], s["k_scale"], phys, off).permute(1, 2, 0).contiguous()
            v = _rows64(s["v_cache"], s["v_scale"], phys, off).permute(1, 0, 2).contiguous()
            late = j[None, :] > (torch.arange(n, device="cuda") + total - n)[:, None]
            bias = torch.zeros(late.shape, dtype=torch.float64, device="cuda")
            bias[late] = -math.inf
            q = s["q"][r0:r0 + n].double().view(n, hkv, grp, -1)
            for head in range(hkv):
                for m in range(grp):
                    logit = (q[:, head, m] @ k[head]) * s["scale"] + bias
                    weight = torch.exp(logit - torch.logsumexp(logit, dim=1, keepdim=True))
                    out[r0:r0 + n, head * grp + m] = weight @ v[head]
        r0 += n
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope_axes_store":
        return _exact_norm_rope_axes_store(s)
    return _exact_attention(s)
