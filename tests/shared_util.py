"""Inputs of the shared-context operators and their plain 64-bit answers."""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import torch

import ops64


def make(groups, H, Hkv, D=128, bs=16, kv="bf16", seed=0, new=None, outside=((), ()), spread=1.0):
    """A batch of groups of sequences: groups = [(prefix_len, [length of each sequence])], where a
    sequence shares its group's whole blocks of the prefix and holds the rest itself (length 0: a
    padding row). outside: lengths of sequences before the first and behind the last group.
    new: new tokens per sequence (None: a decode batch of one query each)."""
    g = torch.Generator().manual_seed(seed)
    lens = [*outside[0], *(n for _, ls in groups for n in ls), *outside[1]]
    cu = [len(outside[0])]
    for _, ls in groups:
        cu.append(cu[-1] + len(ls))
    width = max(1, *(-(-n // bs) for n in lens), *(p // bs for p, _ in groups))
    shared = [min(p, max(ls, default=0)) // bs for p, ls in groups]
    group_of = {b: i for i in range(len(groups)) for b in range(cu[i], cu[i + 1])}
    need = sum(shared) + sum(-(-n // bs) for n in lens)
    nb = need + need // 8 + 2
    perm = torch.randperm(nb, generator=g).tolist()
    heads = [[perm.pop() for _ in range(n)] for n in shared]
    bt = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for j in range(-(-n // bs)):
            head = heads[group_of[b]] if b in group_of else []
            bt[b, j] = head[j] if j < len(head) else perm.pop()
    shape = (nb, bs, Hkv, D)
    s = SimpleNamespace(H=H, Hkv=Hkv, D=D, bs=bs, lens=lens, cu=cu, kv=kv, scale=1 / np.sqrt(D),
                        prefix=[p for p, _ in groups], k_scale=None, v_scale=None, bt=bt.cuda())
    if kv == "bf16":
        s.k_cache, s.v_cache = (torch.randn(shape, generator=g).to(torch.bfloat16).cuda()
                                for _ in range(2))
    else:
        x = [torch.randn(shape, generator=g) for _ in range(2)]
        if kv == "fp8":
            s.k_cache, s.v_cache = ((y * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
                                    .view(torch.uint8).cuda() for y in x)
        else:
            s.k_cache, s.v_cache = ((y * 32).round().clamp(-127, 127).to(torch.int8).cuda()
                                    for y in x)
        one = 1 / (100 if kv == "fp8" else 32)
        s.k_scale, s.v_scale = (one * (0.5 + torch.rand((nb, Hkv, bs), generator=g)).cuda()
                                for _ in range(2))
    rows = len(lens) if new is None else sum(new)
    s.q = (torch.randn((rows, H, D), generator=g) * spread).to(torch.bfloat16).cuda()
    i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32)).cuda()
    s.context_lens, s.cu_groups, s.prefix_lens = i32(lens), i32(cu), i32(s.prefix)
    if new is not None:
        s.new = new
        s.cu_q, s.cu_k = i32(np.concatenate([[0], np.cumsum(new)])), i32(
            np.concatenate([[0], np.cumsum(lens)]))
    return s


def n64(t):
    return t.float().cpu().double().numpy()


def values(s):
    return [ops64.cache_values(c.cpu(), None if sc is None else sc.cpu())
            for c, sc in ((s.k_cache, s.k_scale), (s.v_cache, s.v_scale))]


def decode64(s):
    """Decode attention of every sequence over its own block table row, in 64 bits."""
    kc, vc = values(s)
    q, bt, out = n64(s.q), s.bt.cpu().numpy(), np.zeros(s.q.shape)
    G = s.H // s.Hkv
    for b, n in enumerate(s.lens):
        if n == 0:
            continue
        j = np.arange(n)
        k, v = kc[bt[b][j // s.bs], j % s.bs], vc[bt[b][j // s.bs], j % s.bs]
        for h in range(s.H):
            out[b, h] = ops64.softmax(k[:, h // G] @ q[b, h] * s.scale) @ v[:, h // G]
    return out


def prefill64(s):
    """Causal attention of the new tokens (a window no sequence reaches past), in 64 bits."""
    kc, vc = values(s)
    return ops64.prefill_window(n64(s.q), kc, vc, s.bt.cpu().numpy(), s.cu_q.cpu().numpy(),
                                s.cu_k.cpu().numpy(), s.scale, 1 << 30, 0)
