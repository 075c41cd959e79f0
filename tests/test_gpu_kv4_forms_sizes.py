"""Rotary append, windowed and shared attention at sizes where something else counts: pages past
32-bit offsets, more sequences than a block has threads or keeps the lengths of, several pieces of
prompts of many row tiles."""
import numpy as np
import pytest

import kv4_forms_reference as forms
from gpu_helpers import torch
from test_gpu_kv4 import DT, Setup, cuda, i32, rand_trees
from test_gpu_kv4_rotary import angles, block
from test_gpu_kv4_window import attend, queries

pytestmark = pytest.mark.gpu


def test_pages_far_apart(gpu_lib):
    """Pages 2 GiB apart, so that the last ones lie past 32 bits, against packed ones: the same
    bytes and the same bits."""
    rng, t = np.random.default_rng(0), torch()
    H, Hq, D, P, N = 2, 6, 128, 64, 5
    s = Setup(rng, [150, 149, 140], H, D, P)
    s.pages[..., 32 * D:] = rng.integers(0x20, 0x30, s.pages[..., 32 * D:].shape)
    kw = s.gpu()
    step = 1 << 31
    room = t.empty(len(s.pages) * step, dtype=t.uint8, device="cuda")
    far = room.as_strided(s.g_pages.shape, (step, *s.g_pages.stride()[1:]))
    far.copy_(s.g_pages)
    assert s.table.max() * step > 1 << 33
    table = s.g_table.clone()
    table[1:, 0] = table[0, 0]           # two pages in common: a whole tile
    table[1:, 1] = table[0, 1]
    wide = t.full((3, (1 << 20) // P), -1, dtype=t.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q, k, v = block(rng, 3, N, Hq, H, D, "bf16")
    pos, cs = rng.integers(0, 90, (2, 3, N)), angles(rng, 90, 32)
    axis = cuda(rng.integers(0, 2, 32).astype(np.uint8))
    ws = t.empty(max(gpu_lib.gdn_kv4_attention_workspace_bytes(3, N, Hq, H, D),
                     gpu_lib.gdn_kv4_attention_shared_workspace_bytes(3, N, Hq, H, D, 1)),
                 dtype=t.uint8, device="cuda")
    got = []
    for pages in (s.g_pages, far):
        turned = t.empty(q.shape, dtype=q.dtype, device="cuda")
        gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), cuda(cs), pages, s.g_table, s.g_len,
                                      turned, axis=axis, **kw)
        outs = [turned]
        for call, args, more in ((gpu_lib.gdn_kv4_attention, (), {}),
                                 (gpu_lib.gdn_kv4_attention_window, (), dict(window=70, sinks=5)),
                                 (gpu_lib.gdn_kv4_attention_shared, (i32([0, 3]),), {})):
            o = t.empty_like(turned)
            call(turned, pages, wide, s.g_len, *args, o, ws, scale=0.1, **kw, **more)
            outs.append(o)
        got.append(outs)
    assert int(s.status.item()) == 0
    assert t.equal(far.contiguous(), s.g_pages)
    for a, b in zip(*got):
        assert t.equal(a, b) and a.abs().sum() > 0


@pytest.mark.parametrize("B, N, tree", [(500, 1, False), (600, 3, True), (1100, 2, False),
                                        (1030, 3, True)])
def test_window_of_many_sequences(gpu_lib, B, N, tree):
    rng = np.random.default_rng(B)
    s = Setup(rng, rng.integers(0, 140, B), 1, 64, 32)
    cache = s.fill(rng)
    parent = rand_trees(rng, B, N) if tree else None
    q = queries(rng, B, N, 2, 64, "f16")
    o, lse = attend(gpu_lib, s, q, 33, 2, parent)
    assert int(s.status.item()) == 0
    want = forms.attention(cache, s.table, s.lens, 32, q.double().cpu().numpy(), 64 ** -0.5, s.ks,
                           s.vs, lambda b, n: forms.visible(
                               n, N, None if parent is None else parent[b], 33, 2))
    forms.check(o, lse, want, 140, DT["f16"][1], 64)


@pytest.mark.parametrize("window, sinks", [(60, 5), (200, 0), (1000, 0)])
def test_window_of_several_pieces(gpu_lib, window, sinks):
    """Pieces of three prompts, 21 row tiles each; one of them fills its sequence, one has nodes
    that do not exist."""
    rng = np.random.default_rng(window)
    s = Setup(rng, [691, 333, 300], 2, 64, 96)
    cache = s.fill(rng)
    q = queries(rng, 3, 333, 12, 64, "bf16")
    o, lse = attend(gpu_lib, s, q, window, sinks)
    assert int(s.status.item()) == 0
    want = forms.attention(cache, s.table, s.lens, 96, q.double().cpu().numpy(), 64 ** -0.5, s.ks,
                           s.vs, lambda b, n: forms.visible(n, 333, None, window, sinks))
    forms.check(o, lse, want, 691, DT["bf16"][1], 64)
