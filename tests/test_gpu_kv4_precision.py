"""Attention over the 4-bit cache where single positions carry the result."""
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
