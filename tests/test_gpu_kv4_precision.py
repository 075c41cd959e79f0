"""Attention over the 4-bit cache where single positions carry the result: a large logit
over a long flat tail, and one position of every tile."""
import numpy as np
import pytest

from gpu_helpers import torch
from test_gpu_kv4 import Setup, i32, tdtype

pytestmark = pytest.mark.gpu

ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.mark.parametrize("dtype, T, gap, B, N, Hq, D", [
    # enough sequences that a block has most of an item or all of it
    ("f16", 700, 12, 400, 1, 4, 64),
    ("f16", 4096, 14, 160, 1, 6, 256),
    ("f16", 30000, 18, 160, 1, 4, 128),
    ("bf16", 20000, 16, 160, 8, 6, 128),        # 48 rows
    ("bf16", 9000, 17, 160, 24, 4, 256),        # 96 rows: one scale for all
    ("f16", 131072, 17, 200, 1, 4, 64),
    ("f16", 30000, 18, 1, 1, 4, 128),           # one sequence: a tile or two a block
])
def test_one_large_logit_over_a_flat_tail(gpu_lib, dtype, T, gap, B, N, Hq, D):
    """A first token with a logit `gap` above the others and a value of 0 (an attention sink):
    the output is made of the small probabilities alone.  Each is a binary16 number, 2^7 times
    its share of the row's largest: 2^-11 relative, or 2^-32 of the largest where that is
    more; the other terms as in a flat softmax (fp32 logits and sums, one output rounding)."""
    rng, t = np.random.default_rng(T + D), torch()
    s = Setup(rng, [T], 1, D, 128, ones=True)
    kw = s.gpu()
    gen = t.Generator(device="cuda").manual_seed(T + N)
    u = t.randint(0, 2, (D,), generator=gen, device="cuda") * 2.0 - 1.0
    scale = D ** -0.5
    k = 0.25 * t.randn(1, T, 1, D, generator=gen, device="cuda")
    v = 0.5 + 0.25 * t.randn(1, T, 1, D, generator=gen, device="cuda")
    k[0, 0, 0], v[0, 0, 0] = gap / (scale * D) * u, 0
    gpu_lib.gdn_kv4_append(k, v, s.g_pages, s.g_table, s.g_len, **kw)
    gpu_lib.gdn_kv4_read(s.g_pages, s.g_table, s.g_len, k, v, **kw)   # the stored values
    q = (u + 0.1 * t.randn(B, N, Hq, D, generator=gen, device="cuda")).to(tdtype(dtype))
    table = s.g_table.expand(B, -1).contiguous()     # all sequences hold the same pages
    lens = i32([T] * B)
    o, lse = t.empty_like(q), t.empty(B, N, Hq, device="cuda")
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(B, N, Hq, 1, D), dtype=t.uint8,
                 device="cuda")
    gpu_lib.gdn_kv4_attention(q, s.g_pages, table, lens, o, ws, scale=scale, lse=lse, **kw)
    assert int(s.status.item()) == 0
    kd, vd = k[0, :, 0].double(), v[0, :, 0].double()
    hide = t.arange(T, device="cuda")[None] > T - N + t.arange(N, device="cuda")[:, None]
    for b0 in range(0, B, 20):
        for h in range(Hq):
            x = q[b0:b0 + 20, :, h].double() @ kd.T * scale
            x = x.masked_fill(hide, -float("inf"))
            p = t.exp(x - x.amax(-1, keepdim=True))
            total = p.sum(-1, keepdim=True)
            want, weight = p @ vd / total, p @ vd.abs() / total
            loss = (2.0 ** -11 * p).clamp(min=2.0 ** -32).masked_fill(hide, 0.0) @ vd.abs() / total
            reach = scale * (q[b0:b0 + 20, :, h].double().abs() @ kd.abs().T).amax(-1, keepdim=True)
            d = (D * 2.0 ** -23 + 2.0 ** -20) * reach + 2.0 ** -20
            tol = (ROUND[dtype] * want.abs() + loss + weight * (2 * d + T * 2.0 ** -23)
                   + 2.0 ** -25)
            err = (o[b0:b0 + 20, :, h].double() - want).abs()
            assert bool((err <= tol).all()), f"{float((err / tol).max()):.3f} of the bound"
            l = x.amax(-1) + t.log(total[..., 0])
            assert bool(((lse[b0:b0 + 20, :, h].double() - l).abs()
                         <= d[..., 0] + T * 2.0 ** -23 + 2.0 ** -22 * l.abs()).all())


@pytest.mark.parametrize("dtype, lens, N, Hq, H, D, P", [
    ("bf16", [40000], 1, 6, 1, 256, 64),
    ("bf16", [9000] * 3 + [20011], 16, 12, 2, 256, 64),
    ("f16", [3000 + 7 * i for i in range(40)], 1, 16, 4, 64, 32),
    ("bf16", [2500], 900, 6, 1, 128, 128),
    ("f16", [130 + i for i in range(300)], 1, 8, 2, 128, 32),
    ("bf16", [30011], 22, 6, 1, 128, 96),
])
def test_every_tile_counts(gpu_lib, dtype, lens, N, Hq, H, D, P):
    """One position of every 128 has a logit 30 above the rest (the first or last of its tile
    or any, and the sequence's last): the output is the mean of their values.  Their products
    are exact in fp32 and equal, so the probabilities are one binary16 number (2^-11) and the
    values, small whole numbers, add up exactly; the rest weighs T e^-30.  A tile that is left
    out, counted twice or joined with another weight is far outside the bound: checked for a
    tile left out."""
    rng, t = np.random.default_rng(len(lens) * N + D), torch()
    s = Setup(rng, lens, H, D, P, ones=True)
    kw = s.gpu()
    B, T, G = len(lens), max(lens), Hq // H
    marks = []
    k = np.full((B, T, H), -0.75, np.float32)
    v = rng.choice([-4.0, -2.0, -1.0, 1.0, 2.0, 3.0], (B, T, H, D)).astype(np.float32)
    v[..., ::16] = rng.choice([-6.0, 6.0], (B, T, H, D // 16))        # a scale of exactly 1
    for b, n in enumerate(lens):
        first = 128 * np.arange(-(-n // 128))
        at = first + rng.choice([0, 127, 31, 32, 64, 95], len(first))
        at = np.minimum(at, n - 1)
        marks.append(at)
        k[b, T - n + at] = 0.75
    kt = t.from_numpy(np.ascontiguousarray(np.broadcast_to(k[..., None], (B, T, H, D)))).cuda()
    gpu_lib.gdn_kv4_append(kt, t.from_numpy(v).cuda(), s.g_pages, s.g_table, s.g_len, **kw)
    gain = rng.choice([1.0, 1.25, 1.5], (B, N, Hq))
    q = t.from_numpy(np.ascontiguousarray(np.broadcast_to(gain[..., None], (B, N, Hq, D))))
    q = q.to(tdtype(dtype)).cuda()
    scale = 20.0 / D                                                  # +15 and -15 at gain 1
    o, lse = t.empty_like(q), t.empty(B, N, Hq, device="cuda")
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(B, N, Hq, H, D), dtype=t.uint8,
                 device="cuda")
    gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=scale, lse=lse, **kw)
    assert int(s.status.item()) == 0
    got, glse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        last = n - N + np.arange(N)                                   # a node sees up to here
        count = np.searchsorted(marks[b], last, side="right")         # marks that it sees
        for h in range(H):
            vm = v[b, T - n + marks[b], h].astype(np.float64)
            sums = np.concatenate((np.zeros((1, D)), vm.cumsum(0)))[count]
            has = count > 0
            want = sums / np.maximum(count, 1)[:, None]
            rest = 6 * (T + 1) * np.exp(-30.0)
            tol = (ROUND[dtype] + 2.0 ** -11 + T * 2.0 ** -24) * np.abs(want) + rest + 2.0 ** -25
            for g in range(h * G, h * G + G):
                err = np.abs(got[b, :, g] - want)[has]
                assert (err <= tol[has]).all(), f"{(err / tol[has]).max():.2f} of the bound"
                x = 15.0 * gain[b, :, g]
                l = (x + np.log(np.maximum(count, 1)))[has]
                ltol = rest + T * 2.0 ** -24 + 2.0 ** -20 * l
                assert (np.abs(glse[b, :, g][has] - l) <= ltol).all()
            if count[-1] < 2:
                continue
            # the last node's output without any one of its tiles
            less = (sums[-1] - vm[:count[-1]]) / (count[-1] - 1)
            assert (np.abs(less - want[-1]).max(1) > 2 * tol[-1].max()).all()
