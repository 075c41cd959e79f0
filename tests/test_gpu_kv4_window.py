"""Attention over the 4-bit cache through a window with sinks, on the GPU against 64 bits."""
import numpy as np
import pytest

import kv4_forms_reference as forms
import kv4_reference as ref
from gpu_helpers import torch
from test_gpu_kv4 import DT, Setup, i32, rand_trees, tdtype

pytestmark = pytest.mark.gpu


def queries(rng, B, N, Hq, D, dtype):
    t = torch()
    qkv = t.from_numpy(rng.standard_normal((B, N, (Hq + 2) * D))).cuda().to(tdtype(dtype))
    return qkv[..., :Hq * D].unflatten(-1, (Hq, D))


def attend(gpu_lib, s, q, window, sinks, parent=None):
    t = torch()
    B, N, Hq, D = q.shape
    kw = s.gpu()
    o = t.full((B, N, Hq, D), 5.0, dtype=q.dtype, device="cuda")
    lse = t.full((B, N, Hq), 5.0, device="cuda")
    ws = t.full((gpu_lib.gdn_kv4_attention_workspace_bytes(B, N, Hq, s.H, D),), 255,
                dtype=t.uint8, device="cuda")
    par = None if parent is None else i32(parent)
    for _ in range(2):   # the workspace as a call leaves it serves the next one
        gpu_lib.gdn_kv4_attention_window(q, s.g_pages, s.g_table, s.g_len, o, ws,
                                         scale=D ** -0.5, window=window, sinks=sinks, parent=par,
                                         lse=lse, **kw)
    return o, lse


CASES = [
    # dtype, lens, N, Hq, H, D, P, tree, window, sinks
    ("bf16", [1], 1, 1, 1, 64, 32, False, 1, 0),
    ("bf16", [700], 1, 24, 4, 256, 64, False, 1, 0),
    ("bf16", [700], 1, 24, 4, 256, 64, False, 129, 4),
    ("f16", [0, 1, 31, 129, 300, 640], 1, 8, 2, 128, 32, False, 127, 1),
    ("bf16", [900, 513, 514, 512], 1, 6, 1, 64, 96, False, 128, 130),   # sinks end in a tile
    ("bf16", [900, 385], 1, 6, 2, 128, 64, False, 256, 0),              # whole tiles
    ("bf16", [16, 17, 150, 600], 16, 12, 2, 256, 128, False, 5, 33),    # shorter than the block
    ("f16", [5, 0, 22, 460], 16, 8, 8, 128, 64, False, 64, 3),          # blocks with absent nodes
    ("bf16", [22, 150, 713], 22, 24, 4, 256, 64, True, 100, 4),
    ("f16", [64, 65, 500], 64, 4, 4, 64, 32, True, 3, 0),               # shorter than the paths
    ("f16", [64, 65, 500], 64, 4, 4, 64, 32, True, 7, 68),              # sinks end in the block
    ("bf16", [3, 40, 0], 7, 16, 2, 128, 96, True, 2, 1),                # trees with absent nodes
    ("bf16", [300], 300, 6, 2, 256, 64, False, 50, 10),                 # a prompt from nothing
    ("f16", [691], 333, 10, 2, 128, 1664, False, 200, 0),
    ("bf16", [650], 390, 3, 1, 64, 32, False, 1, 1),
    ("f16", [1000, 40], 2, 34, 2, 128, 64, False, 300, 300),            # two row tiles
    ("bf16", [700, 90], 3, 6, 2, 64, 32, False, 2 ** 31 - 1, 2 ** 31 - 1),
]


@pytest.mark.parametrize("dtype, lens, N, Hq, H, D, P, tree, window, sinks", CASES)
def test_window(gpu_lib, dtype, lens, N, Hq, H, D, P, tree, window, sinks):
    rng = np.random.default_rng(sum(lens) + N * D + Hq + window % 1000)
    s = Setup(rng, lens, H, D, P)
    cache = s.fill(rng)
    parent = rand_trees(rng, len(lens), N) if tree else None
    q = queries(rng, len(lens), N, Hq, D, dtype)
    o, lse = attend(gpu_lib, s, q, window, sinks, parent)
    assert int(s.status.item()) == 0
    want = forms.attention(cache, s.table, s.lens, P, q.double().cpu().numpy(), D ** -0.5, s.ks,
                           s.vs, lambda b, n: forms.visible(
                               n, N, None if parent is None else parent[b], window, sinks))
    forms.check(o, lse, want, max(1, max(lens)), DT[dtype][1], D)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("sinks", [0, 31, 32, 33, 64, 97, 128, 161])
def test_sinks_and_window_share_tiles(gpu_lib, sinks, tree):
    """The window's records follow the sinks' at any place of a tile; pages of 96 tokens end
    inside it, and what lies between is not there."""
    rng = np.random.default_rng(1000 + sinks + tree)
    lens, N, P, window = [1000, 999, 231, 40, 683], 5, 96, 77
    s = Setup(rng, lens, 2, 128, P)
    cache = s.fill(rng)
    parent = rand_trees(rng, len(lens), N) if tree else None
    q = queries(rng, len(lens), N, 6, 128, "bf16")
    table = s.table.copy()
    for b, L in enumerate(lens):
        for j in range(s.width):
            if j * P >= sinks and (j + 1) * P <= L - N - window + 1:
                s.table[b, j] = -1
    o, lse = attend(gpu_lib, s, q, window, sinks, parent)
    assert int(s.status.item()) == 0
    want = forms.attention(cache, table, s.lens, P, q.double().cpu().numpy(), 128 ** -0.5, s.ks,
                           s.vs, lambda b, n: forms.visible(
                               n, N, None if parent is None else parent[b], window, sinks))
    forms.check(o, lse, want, max(lens), DT["bf16"][1], 128)


@pytest.mark.parametrize("N, tree", [(1, False), (40, False), (13, True)])
def test_a_window_as_long_as_the_sequence(gpu_lib, N, tree):
    rng, t = np.random.default_rng(N), torch()
    s = Setup(rng, [500, 333, 41], 2, 128, 64)
    s.fill(rng)
    parent = rand_trees(rng, 3, N) if tree else None
    q = queries(rng, 3, N, 6, 128, "bf16")
    o, lse = attend(gpu_lib, s, q, 500, 0, parent)
    full, flse = t.empty_like(o), t.empty_like(lse)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(3, N, 6, 2, 128), dtype=t.uint8,
                 device="cuda")
    gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, full, ws, scale=128 ** -0.5,
                              parent=None if parent is None else i32(parent), lse=flse,
                              k_scale=s.g_ks, v_scale=s.g_vs)
    assert t.equal(o, full) and t.equal(lse, flse)


@pytest.mark.parametrize("N", [1, 6])
def test_what_no_row_sees_is_not_read(gpu_lib, N):
    """Pages between the sinks and the window may be gone (they are given back), and records of
    their tiles that no row sees hold anything: not read, not reported, the same result."""
    rng, t = np.random.default_rng(20 + N), torch()
    L, P, window, sinks = 1500, 32, 300, 40
    s = Setup(rng, [L], 2, 256, P)
    cache = s.fill(rng)
    q = queries(rng, 1, N, 12, 256, "bf16")
    o, lse = attend(gpu_lib, s, q, window, sinks)
    before = s.table.copy()
    first = L - N - window + 1          # the first node's first
    for j in range(s.width):
        if j * P >= sinks and j * P + P <= first:
            s.table[0, j] = -1
    assert (s.table != before).sum() > 20
    o2, lse2 = attend(gpu_lib, s, q, window, sinks)
    assert int(s.status.item()) == 0 and t.equal(o, o2) and t.equal(lse, lse2)
    want = forms.attention(cache, before, [L], P, q.double().cpu().numpy(), 256 ** -0.5, s.ks, s.vs,
                           lambda b, n: forms.visible(n, N, None, window, sinks))
    forms.check(o2, lse2, want, L, DT["bf16"][1], 256)
    # one page of the window gone: reported, its positions left out
    s.table[0, (L - 100) // P] = 1 << 20
    o3, lse3 = attend(gpu_lib, s, q, window, sinks)
    assert int(s.status.item()) == gpu_lib.GDN_ERR_PAGE_RANGE

    def seen(b, n):
        x = forms.visible(n, N, None, window, sinks)
        x[:, (L - 100) // P * P:((L - 100) // P + 1) * P] = False
        return x
    want = forms.attention(cache, before, [L], P, q.double().cpu().numpy(), 256 ** -0.5, s.ks, s.vs,
                           seen)
    forms.check(o3, lse3, want, L, DT["bf16"][1], 256)


def test_one_large_logit_just_outside_the_window(gpu_lib):
    """A key that would take all the weight lies one position before the window, and is the
    window's first a node earlier."""
    rng, t = np.random.default_rng(31), torch()
    D, L, window = 64, 400, 150
    s = Setup(rng, [L], 1, D, 32, ones=True)
    q = queries(rng, 1, 2, 1, D, "bf16")
    q[0, 1] = q[0, 0]
    cache = s.fill(rng)
    p = L - 2 - window + 1              # the first that node 0 sees; node 1 does not
    kc, ks = ref.quantise(6 * q[0, 0].double().cpu().numpy(), s.ks)
    vc, vs = ref.quantise(np.full((1, D), 3.0), s.vs)
    cache.put(s.table[0, p // 32], 0, p % 32, kc[0], ks[0], vc[0], vs[0])
    o, lse = attend(gpu_lib, s, q, window, 0)
    want = forms.attention(cache, s.table, [L], 32, q.double().cpu().numpy(), D ** -0.5, s.ks, s.vs,
                           lambda b, n: forms.visible(n, 2, None, window, 0))
    assert abs(want[0][0, 0, 0] - 3).max() < 0.1 and abs(want[0][0, 1, 0]).max() < 2
    forms.check(o, lse, want, L, DT["bf16"][1], D)


def test_many_sequences_and_lengths_rewritten(gpu_lib):
    """More sequences than a block keeps the lengths of, in a graph, lengths rewritten between
    replays; one of -1 is skipped and reported."""
    rng, t = np.random.default_rng(32), torch()
    B, D, N = 1100, 64, 2
    lens = rng.integers(0, 60, B)
    s = Setup(rng, lens, 1, D, 32)
    cache = s.fill(rng)
    q = queries(rng, B, N, 2, D, "f16")
    kw = s.gpu()
    o = t.empty(q.shape, dtype=q.dtype, device="cuda")
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(B, N, 2, 1, D), dtype=t.uint8,
                 device="cuda")
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        call = gpu_lib.bind_kv4_attention_window(q, s.g_pages, s.g_table, s.g_len, o, ws,
                                                 scale=D ** -0.5, window=20, sinks=3, **kw)
        call()
        side.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            call()
    for step in range(2):
        if step:
            lens = np.where(rng.random(B) < 0.5, lens, lens // 2)
            lens[7] = -1
            s.g_len.copy_(i32(lens))
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        assert int(s.status.item()) == (gpu_lib.GDN_ERR_ROW_RANGE if step else 0)
        want = forms.attention(cache, s.table, np.maximum(lens, 0), 32, q.double().cpu().numpy(),
                               D ** -0.5, s.ks, s.vs,
                               lambda b, n: forms.visible(n, N, None, 20, 3))
        forms.check(o, None, want, 60, DT["f16"][1], D)


def test_a_bad_tree_is_skipped_and_reported(gpu_lib):
    rng, t = np.random.default_rng(33), torch()
    s = Setup(rng, [300, 300], 1, 64, 32)
    s.fill(rng)
    q = queries(rng, 2, 5, 2, 64, "bf16")
    parent = np.array([[-1, 0, 1, 1, 3], [-1, 0, 1, 1, 3]])
    good, _ = attend(gpu_lib, s, q, 100, 2, parent)
    parent[1, 3] = 3
    o, lse = attend(gpu_lib, s, q, 100, 2, parent)
    assert int(s.status.item()) == gpu_lib.GDN_ERR_BAD_TREE
    assert t.equal(o[0], good[0]) and not o[1].any() and t.isinf(lse[1]).all()
