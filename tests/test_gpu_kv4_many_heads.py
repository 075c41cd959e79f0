"""Attention over the 4-bit cache with more kv heads than the kernels keep the scales of (16), each
with scales of its own, in all forms and head sizes: items written whole, and items joined."""
import numpy as np
import pytest

import kv4_forms_reference as forms
from gpu_helpers import torch
from test_gpu_kv4 import DT, Setup
from test_gpu_kv4_shared import Branches
from test_gpu_kv4_window import attend, queries

pytestmark = pytest.mark.gpu

SIZES = [("bf16", 20, 20, 64, 1), ("f16", 20, 40, 64, 3), ("bf16", 17, 17, 128, 2),
         ("f16", 17, 51, 256, 1), ("bf16", 18, 18, 256, 40)]


@pytest.mark.parametrize("lens", [[60, 100, 33], [1500]])
@pytest.mark.parametrize("dtype, H, Hq, D, N", SIZES)
def test_full_and_window(gpu_lib, dtype, H, Hq, D, N, lens):
    rng, t = np.random.default_rng(H * D + N + len(lens)), torch()
    if D == 256:
        lens = [n // 2 for n in lens]
    s = Setup(rng, lens, H, D, 64)
    s.ks, s.vs = (x.astype(np.float32) for x in (np.geomspace(0.3, 2, H), np.geomspace(4, 0.5, H)))
    cache = s.fill(rng)
    q = queries(rng, len(lens), N, Hq, D, dtype)
    for window, sinks in ((None, 0), (70, 3)):
        if window is None:
            kw = s.gpu()
            o, lse = t.empty_like(q).contiguous(), t.empty(q.shape[:3], device="cuda")
            ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(len(lens), N, Hq, H, D),
                         dtype=t.uint8, device="cuda")
            gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=D ** -0.5,
                                      lse=lse, **kw)
        else:
            o, lse = attend(gpu_lib, s, q, window, sinks)
        assert int(s.status.item()) == 0
        want = forms.attention(cache, s.table, s.lens, 64, q.double().cpu().numpy(), D ** -0.5,
                               s.ks, s.vs, lambda b, n: forms.visible(n, N, None, window, sinks))
        forms.check(o, lse, want, max(lens), DT[dtype][1], D)


@pytest.mark.parametrize("dtype, H, Hq, D, N", SIZES[:4])
def test_shared(gpu_lib, dtype, H, Hq, D, N):
    rng = np.random.default_rng(H * D + N)
    s = Branches(rng, [(3, 4)], [300, 290, 280], H, D, 64)
    s.vs = np.geomspace(4, 0.5, H).astype(np.float32)
    q = queries(rng, 3, N, Hq, D, dtype)
    o, lse = s.attend(gpu_lib, q)
    assert int(s.status.item()) == 0
    forms.check(o, lse, s.want(q), 300, DT[dtype][1], D)
