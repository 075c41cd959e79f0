"""Pages, layers and table rows further apart than they are long, against packed ones."""
import numpy as np
import pytest

from gpu_helpers import torch
from test_gpu_kv4 import Setup, i32, rand_trees, status_word

pytestmark = pytest.mark.gpu


def spread(packed, page_pad, layer_pad):
    """A copy of packed pages [L,n,H,R,36D], each page `page_pad` bytes and each layer
    `layer_pad` bytes further on, in a buffer of 0xA5, and that buffer."""
    t = torch()
    L, n, H, R, rec = packed.shape
    page = H * R * rec + page_pad
    layer = n * page + layer_pad
    room = t.full((L * layer,), 0xA5, dtype=t.uint8, device="cuda")
    view = room.as_strided(packed.shape, (layer, page, R * rec, rec, 1))
    view.copy_(packed)
    return view, room


def padding(room, view):
    t = torch()
    own = t.zeros_like(room, dtype=t.bool)
    own.as_strided(view.shape, view.stride()).fill_(True)
    return room[~own]


def wide(table, more):
    """The table's rows `more` entries further apart; what lies between is no page number."""
    t = torch()
    room = t.full((table.shape[0], table.shape[1] + more), 1 << 29, dtype=t.int32, device="cuda")
    room[:, :table.shape[1]] = table
    return room[:, :table.shape[1]], room


@pytest.mark.parametrize("H, D, P, page_pad, layer_pad, more", [
    (2, 128, 64, 16, 0, 1), (1, 64, 32, 48, 4096, 5), (4, 256, 96, 4096, 32, 3)])
def test_cache_calls(gpu_lib, H, D, P, page_pad, layer_pad, more):
    rng, t = np.random.default_rng(80 + D), torch()
    lens, N = [300, 22, 131], 22
    s = Setup(rng, lens, H, D, P, layers=2)
    kw = s.gpu()
    pages, room = spread(s.g_pages, page_pad, layer_pad)
    table, table_room = wide(s.g_table, more)
    x = t.from_numpy(rng.standard_normal((2, 3, 300, H, D))).cuda().float()
    q = t.from_numpy(rng.standard_normal((3, N, 3 * H, D))).cuda().to(t.bfloat16)
    parent, accept = i32(rand_trees(rng, 3, N)), i32([13, 21, 8])
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(3, N, 3 * H, H, D), dtype=t.uint8,
                 device="cuda")
    outs = []
    for p, tab in ((s.g_pages, s.g_table), (pages, table)):
        o, k, v = t.empty_like(q), t.empty_like(x[0]), t.empty_like(x[0])
        new = i32([0, 0, 0])
        for layer in range(2):
            gpu_lib.gdn_kv4_append(x[layer], x[1 - layer], p[layer], tab, s.g_len, **kw)
        gpu_lib.gdn_kv4_attention(q, p[1], tab, s.g_len, o, ws, scale=0.08, parent=parent, **kw)
        gpu_lib.gdn_kv4_commit(p, tab, s.g_len, accept, new, N=N, parent=parent, status=s.status)
        gpu_lib.gdn_kv4_read(p[1], tab, s.g_len, k, v, **kw)
        outs.append((o, k, v, new, p.clone()))
    assert int(s.status.item()) == 0
    assert all(t.equal(a, b) for a, b in zip(*outs)) and outs[0][0].any()
    assert bool((padding(room, pages) == 0xA5).all())
    assert bool((table_room[:, table.shape[1]:] == 1 << 29).all())


@pytest.mark.parametrize("page_pad, layer_pad, more", [(16, 0, 1), (4096, 4096, 7)])
def test_pool_calls(gpu_lib, page_pad, layer_pad, more):
    rng, t = np.random.default_rng(90), torch()
    H, D, P, n_pages, rows, width = 3, 64, 96, 30, 6, 5
    packed = t.from_numpy(rng.integers(0, 256, (2, n_pages, H, P // 32, 36 * D),
                                       dtype=np.uint8)).cuda()
    pages, room = spread(packed, page_pad, layer_pad)
    states = []
    for p in (packed, pages):
        table = i32(np.full((rows, width), -1))
        if p is pages:
            table, table_room = wide(table, more)
        pool = (table, i32(np.zeros(rows)), i32(np.zeros(n_pages)))
        status = status_word()
        ws = t.empty(gpu_lib.gdn_kv4_reserve_workspace_bytes(rows), dtype=t.uint8, device="cuda")
        gpu_lib.gdn_kv4_reserve(p, *pool, i32([0, 1]), i32([200, 130]), ws, status=status)
        gpu_lib.gdn_kv4_fork(*pool, i32([0, 0, 1]), i32([2, 3, 5]), page_tokens=P, status=status)
        gpu_lib.gdn_kv4_reserve(p, *pool, i32([3, 2, 5]), i32([290, 201, 400]), ws, status=status)
        gpu_lib.gdn_kv4_release(*pool, i32([0, 5]), i32([97, 0]), page_tokens=P, status=status)
        assert int(status.item()) == 0
        states.append((*(x.clone() for x in pool), p.clone()))
    assert all(t.equal(a, b) for a, b in zip(*states))
    assert not t.equal(states[0][3], t.zeros_like(states[0][3]))
    assert int((states[0][2] > 0).sum()) == 7
    assert bool((padding(room, pages) == 0xA5).all())
    assert bool((table_room[:, width:] == 1 << 29).all())
