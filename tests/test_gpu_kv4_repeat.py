"""The attention's bits over the 4-bit cache go with its inputs alone: not with what kernels before
it left in shared memory, tensor memory or the workspace."""
import numpy as np
import pytest

from gpu_helpers import torch
from test_gpu_kv4 import Setup, i32, rand_trees
from test_gpu_kv4_window import queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["full", "window", "shared"])
@pytest.mark.parametrize("N, Hq, H, D, tree", [(1, 8, 2, 128, False), (1, 24, 4, 256, False),
                                               (3, 4, 2, 64, False), (16, 24, 4, 256, False),
                                               (40, 6, 2, 128, False), (9, 8, 2, 128, True)])
def test_bits_do_not_depend_on_what_ran_before(gpu_lib, form, N, Hq, H, D, tree):
    rng, t = np.random.default_rng(60 + N), torch()
    lens = rng.integers(N, 900, 24)
    lens[:6] = [N, 129 + N, 257, 300, 640, 899]
    s = Setup(rng, lens, H, D, 64)
    s.fill(rng)
    kw = s.gpu()
    if form == "shared":   # as wide as a server's table, so that the pages are compared
        wide = t.full((24, 16384), -1, dtype=t.int32, device="cuda")
        wide[:, :s.width] = s.g_table
        s.g_table = wide
    parent = i32(rand_trees(rng, 24, N)) if tree else None
    q = queries(rng, 24, N, Hq, D, "f16")
    size = (24, N, Hq, H, D)
    ws = t.empty(gpu_lib.gdn_kv4_attention_shared_workspace_bytes(*size, 2), dtype=t.uint8,
                 device="cuda")

    def attend(pages):
        o = t.empty_like(q, memory_format=t.contiguous_format)
        lse = t.empty(24, N, Hq, device="cuda")
        args = dict(scale=D ** -0.5, parent=parent, lse=lse, **kw)
        if form == "full":
            gpu_lib.gdn_kv4_attention(q, pages, s.g_table, s.g_len, o, ws, **args)
        elif form == "window":
            gpu_lib.gdn_kv4_attention_window(q, pages, s.g_table, s.g_len, o, ws, window=200,
                                             sinks=5, **args)
        else:
            gpu_lib.gdn_kv4_attention_shared(q, pages, s.g_table, s.g_len, i32([0, 9, 24]), o, ws,
                                             **args)
        return o, lse

    # records whose scales are no numbers, large ones, and zeros, left in shared memory by a call
    # over them before
    want = None
    for fill in (None, 255, 126, 0, None):
        if fill is not None:
            attend(t.full_like(s.g_pages, fill))
            ws.fill_(fill)
        o, lse = attend(s.g_pages)
        if want is None:
            want = o.clone(), lse.clone()
        assert t.equal(o, want[0]) and t.equal(lse, want[1])
    assert int(s.status.item()) == 0
