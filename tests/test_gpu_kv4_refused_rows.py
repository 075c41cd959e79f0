"""A round goes on beside a row that the page pool could not serve: with the granted
lengths of gdn_kv4_reserve, that row and the other holders of its pages stay as they are."""
import os
import sys

import numpy as np
import pytest

from gpu_helpers import torch
from test_gpu_kv4 import i32, status_word

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(gpu_lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import speculative_round
    finally:
        sys.path.pop(0)
    return speculative_round


def stored(gpu_lib, pages, table, row, n, H, D):
    t = torch()
    k, v = (t.empty(1, n, H, D, device="cuda") for _ in range(2))
    gpu_lib.gdn_kv4_read(pages, table[row:row + 1], i32([n]), k, v)
    return k, v


@pytest.mark.parametrize("F", [3, 600])
def test_granted_lengths(gpu_lib, F):
    """new_len for a row that was served, -1 for one that was not, for any number of rows."""
    t, rng = torch(), np.random.default_rng(F)
    P, width, n_pages = 32, 4, F + 1
    table, kv_len, count = i32(np.full((F, width), -1)), i32(np.zeros(F)), i32(np.zeros(n_pages))
    pages = t.zeros(n_pages, 1, 1, 36 * 64, dtype=t.uint8, device="cuda")
    ws = t.empty(gpu_lib.gdn_kv4_reserve_workspace_bytes(F), dtype=t.uint8, device="cuda")
    rows = rng.permutation(F)
    new = rng.integers(1, 2 * P + 1, F)
    new[1] = width * P + 1                      # a length the table has no room for
    granted, status = i32(np.full(F, 7)), status_word()
    gpu_lib.gdn_kv4_reserve(pages, table, kv_len, count, i32(rows), i32(new), ws, status=status,
                            granted=granted)
    got, lens = granted.cpu().numpy(), kv_len.cpu().numpy()[rows]
    asked = np.where(np.arange(F) == 1, 0, -(-new // P))
    served = (np.cumsum(asked) <= n_pages) & (np.arange(F) != 1)
    assert served.any() and not served.all()
    assert np.array_equal(got, np.where(served, new, -1))
    assert np.array_equal(lens, np.where(served, new, 0))
    # a row that asks for nothing new is granted what it has, when no page is free as well
    gpu_lib.gdn_kv4_reserve(pages, table, kv_len, count, i32(rows[:1]), i32(new[:1]), ws,
                            granted=granted[:1])
    assert int(granted[0]) == new[0]


def test_refused_branch_leaves_its_source_and_siblings(gpu_lib):
    """Three branches of one sequence grow; the last finds no page.  Its shared last page,
    which the source and nobody else still reads, keeps its bytes through append and commit."""
    t = torch()
    H, D, P, N = 2, 128, 64, 6
    pages = t.zeros(5, H, P // 32, 36 * D, dtype=t.uint8, device="cuda")
    table, length, count = i32(np.full((4, 4), -1)), i32(np.zeros(4)), i32(np.zeros(5))
    pool = (table, length, count)
    status = status_word()
    ws = t.empty(gpu_lib.gdn_kv4_reserve_workspace_bytes(3), dtype=t.uint8, device="cuda")
    gen = t.Generator(device="cuda").manual_seed(3)
    k0 = t.randn(1, 100, H, D, generator=gen, device="cuda")
    gpu_lib.gdn_kv4_reserve(pages, *pool, i32([0]), i32([100]), ws, status=status)
    gpu_lib.gdn_kv4_append(k0, -k0, pages, table[:1], length[:1], status=status)
    gpu_lib.gdn_kv4_fork(*pool, i32([0, 0, 0]), i32([1, 2, 3]), page_tokens=P, status=status)
    count[4] = 1                                # two free pages are left: 2 and 3
    assert int(status.item()) == 0
    before = stored(gpu_lib, pages, table, 0, 100, H, D)
    rows, granted = i32([1, 2, 3]), i32([0, 0, 0])
    gpu_lib.gdn_kv4_reserve(pages, *pool, rows, i32([100 + N] * 3), ws, status=status,
                            granted=granted)
    assert int(status.item()) == gpu_lib.GDN_ERR_POOL_EMPTY
    assert granted.tolist() == [100 + N, 100 + N, -1]
    assert length.tolist() == [100, 100 + N, 100 + N, 100]
    snapshot, held, row3 = pages.clone(), count.clone(), table[3].clone()
    k = t.randn(3, N, H, D, generator=gen, device="cuda")
    gpu_lib.gdn_kv4_append(k, -k, pages, table[1:], granted, status=status)
    own = table[3, 1:2].long()
    assert t.equal(pages[own], snapshot[own])
    q = t.randn(3, N, 4, D, generator=gen, device="cuda").to(t.bfloat16)
    o = t.full_like(q, 9)
    aws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(3, N, 4, H, D), dtype=t.uint8,
                  device="cuda")
    gpu_lib.gdn_kv4_attention(q, pages, table[1:], granted, o, aws, scale=0.1, status=status)
    assert o[:2].any() and not o[2].any()
    parent = i32([[-1, 0, 0, 2, 3, 3]] * 3)
    committed = i32([0, 0, 0])
    gpu_lib.gdn_kv4_commit(pages, table[1:], granted, i32([4, 1, 4]), committed, N=N,
                           parent=parent, status=status)
    assert committed.tolist() == [104, 102, -1]
    gpu_lib.gdn_kv4_release(*pool, rows, committed, page_tokens=P, status=status)
    assert length.tolist() == [100, 104, 102, 100]
    assert t.equal(count, held) and t.equal(table[3], row3)
    for row in (0, 3):
        for x, y in zip(stored(gpu_lib, pages, table, row, 100, H, D), before):
            assert t.equal(x, y)
    # the served branches hold the old tokens and their own path
    for row, path in ((1, [0, 2, 3, 4]), (2, [0, 1])):
        got, _ = stored(gpu_lib, pages, table, row, 100 + len(path), H, D)
        assert t.equal(got[:, :100], before[0])
        lone, one = t.zeros_like(pages), i32([len(path)])
        x, back = k[row - 1:row, path].contiguous(), t.empty(1, len(path), H, D, device="cuda")
        gpu_lib.gdn_kv4_append(x, x, lone, i32([[0]]), one)
        gpu_lib.gdn_kv4_read(lone, i32([[0]]), one, back, t.empty_like(back))
        assert t.equal(got[0, 100:], back[0])
    assert int(status.item()) == gpu_lib.GDN_ERR_POOL_EMPTY


def test_example_round_with_a_full_pool(example, gpu_lib):
    """The example's sequence that finds no page keeps its tokens, its pages and its
    recurrent state; the other goes on."""
    t = torch()
    m = example.Mixers(2, recurrent=1, N=22, max_tokens=200)
    _, _, _, Hq, Hkv, D = m.shape
    m.prompt(120)                               # pages of 64 tokens: two each
    assert int(m.status.item()) == 0
    m.ref[m.ref == 0] = 1                       # the pool is full but for one page
    m.ref[5] = 0
    host = t.Generator().manual_seed(4)
    parent = example.random_trees(2, 22, host).cuda()
    accept = i32([20, 21])
    before = [stored(gpu_lib, m.pages, m.table, b, 120, Hkv, D) for b in range(2)]
    state, count, row1 = m.state[0].clone(), m.ref.clone(), m.table[1].clone()
    qkv = m.normal(2, 22, (Hq + 2 * Hkv) * D, dtype=t.bfloat16)
    o, _ = m.verify(parent, qkv, [example.recurrent_inputs(m)])
    m.commit(parent, accept)
    assert int(m.status.item()) == gpu_lib.GDN_ERR_POOL_EMPTY
    lens = m.length.tolist()
    assert lens[0] > 120 and lens[1] == 120
    assert o[0].any() and not o[1].any()
    for b in range(2):
        got = stored(gpu_lib, m.pages, m.table, b, 120, Hkv, D)
        assert all(t.equal(x, y) for x, y in zip(got, before[b]))
    assert t.equal(m.table[1], row1)
    assert t.equal(m.ref[row1[row1 >= 0].long()], count[row1[row1 >= 0].long()])
    assert not t.equal(m.state[0][0], state[0]) and t.equal(m.state[0][1], state[1])
