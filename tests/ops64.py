"""Plain 64-bit implementations of the bounded-cache operators, on host arrays.

Written from the formulas with numpy, one sequence and head at a time; nothing
here is shared with the library. Caches are torch CPU tensors as the library
takes them; values are float64 arrays.
"""
from __future__ import annotations

import numpy as np
import torch

FP8_MAX, INT8_MAX = 448.0, 127.0


def cache_values(cache: torch.Tensor, scale: torch.Tensor | None) -> np.ndarray:
    """The cache's values: code * scale for 8-bit caches. (NB, bs, Hkv, D) float64."""
    if cache.dtype == torch.uint8:
        x = cache.view(torch.float8_e4m3fn).float().double().numpy()
    else:
        x = cache.double().numpy()
    return x if scale is None else x * scale.double().permute(0, 2, 1).numpy()[..., None]


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """(y, magnitude): the normalised and rotated heads of x (T, n, D) and, per element, the
    sum of the absolute terms it is made of (for error bounds)."""
    x = np.asarray(x, dtype=np.float64)
    T, n, D = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, mag = x.copy(), np.abs(x)
    if cos_sin is None:
        return y, mag
    rot = cos_sin.shape[1]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c = cos_sin[positions, i].astype(np.float64)[:, None]
        s = cos_sin[positions, rot // 2 + i].astype(np.float64)[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
        mag[:, :, a] = np.abs(x[:, :, a] * c) + np.abs(x[:, :, b] * s)
        mag[:, :, b] = np.abs(x[:, :, b] * c) + np.abs(x[:, :, a] * s)
    return y, mag


def softmax(x):
    e = np.exp(x - x.max(axis=-1, keepdims=True))
    return e / e.sum(axis=-1, keepdims=True)


def prefill_window(q, kc, vc, bt, cu_q, cu_k, scale, window, sinks):
    """q (total, H, D) float64, kc / vc cache values. Rows that see no key are zero."""
    out = np.zeros_like(q)
    bs, hkv = kc.shape[1:3]
    G = q.shape[1] // hkv
    for b in range(len(cu_q) - 1):
        n, kv = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        cached = max(kv - n, 0)
        for i in range(n):
            p = i + cached
            j = np.arange(kv)
            j = j[(j <= p) & ((j < sinks) | (j > p - window))]
            if not len(j):
                continue
            phys, off = bt[b][j // bs], j % bs
            for h in range(q.shape[1]):
                w = softmax(kc[phys, off, h // G] @ q[cu_q[b] + i, h] * scale)
                out[cu_q[b] + i, h] = w @ vc[phys, off, h // G]
    return out


def decode_scored(q, kc, vc, bt, lens, scale, shape):
    """(out, weights added to the scores (NB, Hkv, bs), their error weights): the third array
    is the sum over the heads of weight * sum_i |q_i k_i| * scale (a score's error scale)."""
    out, add, mag = np.zeros_like(q), np.zeros(shape), np.zeros(shape)
    bs, hkv = kc.shape[1:3]
    G = q.shape[1] // hkv
    for b, n in enumerate(lens):
        if n == 0:
            continue
        j = np.arange(n)
        phys, off = bt[b][j // bs], j % bs
        for h in range(q.shape[1]):
            k = kc[phys, off, h // G]
            w = softmax(k @ q[b, h] * scale)
            out[b, h] = w @ vc[phys, off, h // G]
            np.add.at(add, (phys, h // G, off), w)
            np.add.at(mag, (phys, h // G, off), w * (np.abs(k) @ np.abs(q[b, h])).max() * scale)
    return out, add, mag


def evict_rows(scores, bt, lens, budget, sinks, recent):
    """(kept (B, Hkv, budget), new_lens): by sorting the middle keys of every head."""
    hkv, bs = scores.shape[1:]
    kept = np.full((len(lens), hkv, budget), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for g in range(hkv):
            if n <= budget:
                kept[b, g, :n] = np.arange(n)
                continue
            mid = np.arange(sinks, n - recent)
            x = scores[bt[b][mid // bs], g, mid % bs].astype(np.float64)
            x = np.where(np.isnan(x), np.inf, x)
            nan = np.isnan(scores[bt[b][mid // bs], g, mid % bs])
            order = np.lexsort((mid, -x, ~nan))  # NaN first, then the value, then the position
            kept[b, g] = np.sort(np.concatenate([
                np.arange(sinks), mid[order[:budget - sinks - recent]], np.arange(n - recent, n)]))
    return kept, np.minimum(np.asarray(lens, dtype=np.int32), budget)


def move_rows(t, by_slot, kept, bt, lens, budget, bs):
    """A copy of a cache (by_slot: (NB, bs, Hkv, D)) or score / scale array ((NB, Hkv, bs))
    with the kept rows at the front of their sequences."""
    new = t.clone()
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        for g in range(kept.shape[1]):
            for i, p in enumerate(kept[b, g]):
                dst, src = (int(bt[b][i // bs]), i % bs), (int(bt[b][p // bs]), int(p) % bs)
                if by_slot:
                    new[dst[0], dst[1], g] = t[src[0], src[1], g]
                else:
                    new[dst[0], g, dst[1]] = t[src[0], g, src[1]]
    return new
