"""The shared-context operators together, as a server of questions about one video uses them: the
video's tokens (positions on three axes) stored once by norm_rope_axes_store, the questions' tokens
stored behind them and answered over the shared blocks by prefill_shared, then decode steps
(norm_rope_axes_store, decode_shared), every output against plain 64-bit arithmetic on the caches
the library wrote."""
import numpy as np
import pytest
import torch

import ops64
import paged_kv_cache_186_gb300 as pa
from gpu_util import assert_attention_close
from test_norm_rope import check_rows, table

pytestmark = pytest.mark.gpu

AXIS_OF = [0] * 16 + [1] * 24 + [2] * 24


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_questions_about_one_video(kv):
    H, Hkv, D, bs, B, video, steps = 8, 2, 128, 16, 5, 3 * 8 * 9, 6
    questions = [7, 1, 20, 3, 12]
    g = torch.Generator().manual_seed(900)
    nb, width, shared = 64, 18, video // bs
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    bt = torch.empty((B, width), dtype=torch.int32)
    bt[:, :shared] = perm[:shared]
    bt[:, shared:] = perm[shared:shared + B * (width - shared)].view(B, -1)
    bt = bt.cuda()
    if kv == "bf16":
        kc, vc = (torch.full((nb, bs, Hkv, D), float("nan"), dtype=torch.bfloat16).cuda()
                  for _ in range(2))
        ks = vs = None
    else:
        kc, vc = (torch.full((nb, bs, Hkv, D), 0x7f, dtype=torch.uint8).cuda() for _ in range(2))
        ks, vs = (torch.full((nb, Hkv, bs), float("nan")).cuda() for _ in range(2))
    cs = torch.from_numpy(table(256, D)).cuda()
    qw, kw = (1 + 0.2 * torch.randn((2, D), generator=g)).to(torch.bfloat16).cuda()
    scale = 1 / np.sqrt(D)
    cu_groups = torch.tensor([0, B], dtype=torch.int32).cuda()
    prefix = torch.tensor([video], dtype=torch.int32).cuda()
    n64 = lambda t: t.float().cpu().double().numpy()
    tables = bt.cpu().numpy()

    def store(where, pos):
        """New tokens at (sequence, place) `where` with three positions each."""
        T = len(where)
        qkv = torch.randn((T, (H + 2 * Hkv) * D), generator=g).to(torch.bfloat16).cuda()
        q, k, v = (x.view(T, -1, D) for x in qkv.split([H * D, Hkv * D, Hkv * D], dim=1))
        slots = [int(tables[b, p // bs]) * bs + p % bs for b, p in where]
        pos = np.array(pos).T.copy()
        out = pa.norm_rope_axes_store(q, k, v, torch.from_numpy(pos).cuda(),
                                      torch.tensor(slots).cuda(), kc, vc, AXIS_OF, cs, q_weight=qw,
                                      k_weight=kw, k_scale=ks, v_scale=vs)
        own = np.empty((T, D), dtype=np.float32)
        for i, a in enumerate(AXIS_OF):
            own[:, i], own[:, 64 + i] = (cs.cpu().numpy()[pos[a], c] for c in (i, 64 + i))
        want, mag = ops64.norm_rope(n64(q), n64(qw), 1e-6, own, np.arange(T), False)
        check_rows(n64(out), want, mag, "q")
        return out

    def values():
        return [ops64.cache_values(c.cpu(), None if s is None else s.cpu())
                for c, s in ((kc, ks), (vc, vs))]

    # the video: frames of 8 x 9, in the shared blocks (and, behind the last whole one, in each
    # sequence's own); then each question, whose positions go on from the video's largest
    frames = [(p // 72, p // 9 % 8, p % 9) for p in range(video)]
    store([(0, p) for p in range(video)], frames)
    tail = range(shared * bs, video)
    for b in range(1, B):  # the part of a block behind the shared ones
        for p in tail:
            src, dst = (int(tables[0, p // bs]), p % bs), (int(tables[b, p // bs]), p % bs)
            kc[dst], vc[dst] = kc[src].clone(), vc[src].clone()
            if ks is not None:
                ks[dst[0], :, dst[1]], vs[dst[0], :, dst[1]] = (ks[src[0], :, src[1]].clone(),
                                                                vs[src[0], :, src[1]].clone())
    where = [(b, video + i) for b, n in enumerate(questions) for i in range(n)]
    q = store(where, [(9 + i,) * 3 for n in questions for i in range(n)])
    lens = [video + n for n in questions]
    cu = lambda x: torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32).cuda()
    if kv == "bf16":
        out = pa.prefill_shared(q, kc, vc, bt, cu(questions), cu(lens), cu_groups, prefix, scale,
                                max_q_len=max(questions), always=True)
        want = ops64.prefill_window(n64(q), *values(), tables, cu(questions).cpu().numpy(),
                                    cu(lens).cpu().numpy(), scale, 1 << 30, 0)
        assert_attention_close(out, want, "questions")
    for step in range(steps):
        q = store([(b, lens[b]) for b in range(B)], [(9 + questions[b] + step,) * 3 for b in range(B)])
        lens = [n + 1 for n in lens]
        out = pa.decode_shared(q, kc, vc, bt, torch.tensor(lens, dtype=torch.int32).cuda(), cu_groups,
                               prefix, scale, always=True, k_scale=ks, v_scale=vs)
        k64, v64 = values()
        want = np.zeros(q.shape)
        for b, n in enumerate(lens):
            j = np.arange(n)
            for h in range(H):
                k, v = (x[tables[b][j // bs], j % bs, h // (H // Hkv)] for x in (k64, v64))
                want[b, h] = ops64.softmax(k @ n64(q)[b, h] * scale) @ v
        assert_attention_close(out, want, f"step {step}")
    assert pa.get_device_error() == 0
