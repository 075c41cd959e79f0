"""Sequences of the 4-bit cache that cannot be served are left as they are: bad page
numbers, beside sequences that are served."""
import numpy as np
import pytest

import kv4_reference as ref
from gpu_helpers import torch
from test_gpu_kv4 import Setup, i32, status_word

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_commit_on_a_bad_page_leaves_the_sequence(gpu_lib, which, page):
    """One of the block's pages is not there: no layer moves, the length stays, and the
    sequences beside it are committed."""
    rng, t = np.random.default_rng(70 + which), torch()
    N, P, layers = 40, 32, 2
    s = Setup(rng, [90, 90, 131], 2, 64, P, layers=layers)
    s.gpu()
    parent = np.tile([-1, 0, 0] + [2] + list(range(3, N - 1)), (3, 1))   # node 1 is a leaf
    accept = np.array([N - 1, N - 1, 7])
    # sequence 1's block is at 50 .. 89: pages 1 and 2 of its row; which = 0: a page before
    # the block, which the call has no business with
    s.g_table[1, which] = page
    out = i32([-7, -7, -7])
    before = s.g_pages.clone()
    gpu_lib.gdn_kv4_commit(s.g_pages, s.g_table, s.g_len, i32(accept), out, N=N,
                           parent=i32(parent), status=s.status)
    want = ref.commit([ref.Cache(s.pages[l], 64) for l in range(layers)], s.table, s.lens, P, N,
                      accept, parent)
    assert int(s.status.item()) == (gpu_lib.GDN_ERR_PAGE_RANGE if which else 0)
    if which:
        want[1] = 90
    assert out.tolist() == want.tolist()
    own = s.table[1][s.table[1] >= 0]
    if which:
        assert t.equal(s.g_pages[:, own], before[:, own])
    got = s.g_pages.cpu().numpy()
    for l in range(layers):
        a, b_ = ref.Cache(got[l], 64), ref.Cache(s.pages[l], 64)
        for b in (0, 2) if which else (0, 1, 2):
            for p in range(int(want[b])):
                for h in range(2):
                    for x, y in zip(a.get(s.table[b, p // P], h, p % P),
                                    b_.get(s.table[b, p // P], h, p % P)):
                        assert np.array_equal(x, y)


def test_commit_with_nothing_to_move_does_not_look_at_the_pages(gpu_lib):
    """A chain, and a tree's path that is in place, are committed by their length alone."""
    rng = np.random.default_rng(75)
    s = Setup(rng, [40], 1, 64, 32)
    s.gpu()
    s.g_table[0] = -1
    for parent in (None, i32([[-1, 0, 1, 2]])):
        out = i32([0])
        gpu_lib.gdn_kv4_commit(s.g_pages, s.g_table, s.g_len, i32([2]), out, N=4, parent=parent,
                               status=s.status)
        assert out.tolist() == [39] and int(s.status.item()) == 0


# ------------------------------------------------------------------ pool
def pool_of(widths, P=32, width=200, rows=8):
    """Rows of `widths` pages each, their last page partly filled, then empty rows."""
    table, kv_len = np.full((rows, width), -1, np.int64), np.zeros(rows, np.int64)
    at = 0
    for r, w in enumerate(widths):
        table[r, :w] = np.arange(at, at + w)
        kv_len[r] = w * P - 5
        at += w
    count = np.zeros(at + 40, np.int64)
    count[:at] = 1
    return ref.Pool(table, kv_len, count, P)


BAD = [(3, -1), (3, 1 << 20), (0, -5), (150, -1), (180, 1 << 20)]   # entry, page number


@pytest.mark.parametrize("entry, page", BAD)
def test_fork_of_a_row_with_a_bad_page_leaves_everything(gpu_lib, entry, page):
    t = torch()
    pool = pool_of([190, 5])
    g = [i32(pool.table), i32(pool.kv_len), i32(pool.ref)]
    g[0][0, entry] = page
    row0 = g[0][0].clone()
    pool.fork([1], [5])
    status = status_word()
    gpu_lib.gdn_kv4_fork(*g, i32([0, 1]), i32([4, 5]), page_tokens=32, status=status)
    assert int(status.item()) == gpu_lib.GDN_ERR_PAGE_RANGE
    assert t.equal(g[0][0], row0)
    assert np.array_equal(g[0][1:].cpu().numpy(), pool.table[1:])
    assert np.array_equal(g[1].cpu().numpy(), pool.kv_len)
    assert np.array_equal(g[2].cpu().numpy(), pool.ref)


@pytest.mark.parametrize("entry, page", BAD)
def test_release_of_a_row_with_a_bad_page_leaves_everything(gpu_lib, entry, page):
    t = torch()
    pool = pool_of([190, 5])
    g = [i32(pool.table), i32(pool.kv_len), i32(pool.ref)]
    g[0][0, entry] = page
    row0 = g[0][0].clone()
    pool.release([1], [40])
    status = status_word()
    gpu_lib.gdn_kv4_release(*g, i32([0, 1]), i32([0, 40]), page_tokens=32, status=status)
    assert int(status.item()) == gpu_lib.GDN_ERR_PAGE_RANGE
    assert t.equal(g[0][0], row0)
    assert np.array_equal(g[0][1:].cpu().numpy(), pool.table[1:])
    assert np.array_equal(g[1].cpu().numpy(), pool.kv_len)
    assert np.array_equal(g[2].cpu().numpy(), pool.ref)


def test_release_past_a_bad_page_is_served(gpu_lib):
    """Only the pages that are given up have to be there."""
    pool = pool_of([190])
    g = [i32(pool.table), i32(pool.kv_len), i32(pool.ref)]
    g[0][0, 3] = -1
    pool.table[0, 3] = -1
    pool.release([0], [200])
    status = status_word()
    gpu_lib.gdn_kv4_release(*g, i32([0]), i32([200]), page_tokens=32, status=status)
    assert int(status.item()) == 0
    for got, want in zip(g, (pool.table, pool.kv_len, pool.ref)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("page", [-1, 1 << 20])
def test_reserve_on_a_bad_last_page_leaves_the_row(gpu_lib, page):
    t = torch()
    pool = pool_of([4, 5])
    g = [i32(pool.table), i32(pool.kv_len), i32(pool.ref)]
    g[0][0, 3] = page
    row0 = g[0][0].clone()
    assert pool.reserve([1], [170]) == []
    pages = t.zeros(len(pool.ref), 1, 1, 36 * 64, dtype=t.uint8, device="cuda")
    ws = t.empty(gpu_lib.gdn_kv4_reserve_workspace_bytes(2), dtype=t.uint8, device="cuda")
    status = status_word()
    gpu_lib.gdn_kv4_reserve(pages, *g, i32([0, 1]), i32([130, 170]), ws, status=status)
    assert int(status.item()) == gpu_lib.GDN_ERR_PAGE_RANGE
    assert t.equal(g[0][0], row0)
    assert np.array_equal(g[0][1:].cpu().numpy(), pool.table[1:])
    assert np.array_equal(g[1].cpu().numpy(), pool.kv_len)
    assert np.array_equal(g[2].cpu().numpy(), pool.ref)
