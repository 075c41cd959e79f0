"""What the plan of the attention over shared pages decides, on the GPU against a plain count:
results alone cannot tell whether anything was shared.  The plan is the workspace's first three
arrays (256-byte steps), groups and then sequences in each: lengths, a group's members or a
sequence's first own tile (-1: skipped), first sequence and table row (16 bits each)."""
import numpy as np
import pytest

from gpu_helpers import torch
from test_gpu_kv4 import cuda, i32, status_word

pytestmark = pytest.mark.gpu

TILE, WIDE = 128, 1 << 20   # tokens of a tile; of a table that is wide enough for sharing to pay


class Batch:
    """Sequences over pages of random codes (scales of 2^-3 and 2^-2: values of at most 1.5).
    groups: (members, pages in common); the rest of a row are pages of its own."""

    def __init__(self, rng, groups, lens, P, H=1, D=64):
        self.P, self.H, self.D, self.lens = P, H, D, np.asarray(lens)
        held = [max(0, -(-int(n) // P)) for n in lens]
        self.table = np.full((len(lens), WIDE // P), -1, np.int32)
        at, b, self.group = 0, 0, [0]
        for members, common in groups:
            start, at = at, at + common
            for _ in range(members):
                n = min(common, held[b])
                self.table[b, :n] = np.arange(start, start + n)
                self.table[b, n:held[b]] = np.arange(at, at + held[b] - n)
                at += held[b] - n
                b += 1
            self.group.append(b)
        self.pages = rng.integers(0, 256, (at + 1, H, P // 32, 36 * D), dtype=np.uint8)
        self.pages[..., 32 * D:] = rng.choice(np.array([0x20, 0x28], np.uint8),
                                                 self.pages[..., 32 * D:].shape)

    def run(self, gpu_lib, N=1, Hq=1, parent=None):
        """The plan's numbers, the status, and outputs of the shared and the full attention."""
        t = torch()
        B, G = len(self.lens), len(self.group) - 1
        q = t.randn((B, N, Hq, self.D), generator=t.Generator("cuda").manual_seed(B + N),
                    device="cuda").half()
        size = gpu_lib.gdn_kv4_attention_shared_workspace_bytes(B, N, Hq, self.H, self.D, G)
        ws = t.full((size,), 255, dtype=t.uint8, device="cuda")
        pages, table, lens = cuda(self.pages), i32(self.table), i32(self.lens)
        status, par = status_word(), None if parent is None else i32(parent)
        o, want = t.empty_like(q), t.empty_like(q)
        kw = dict(scale=self.D ** -0.5, parent=par)
        gpu_lib.gdn_kv4_attention_shared(q, pages, table, lens, i32(self.group), o, ws,
                                         status=status, **kw)
        step = -(-4 * (G + B) // 256) * 256
        plan = [ws[i * step:i * step + 4 * (G + B)].view(t.int32).cpu().numpy() for i in range(3)]
        gpu_lib.gdn_kv4_attention(q, pages, table, lens, want, ws, status=status_word(), **kw)
        return plan, int(status.item()), (o, want, q, max(self.lens))

    def expect(self, N=1, skipped=()):
        """Groups' shared lengths and members, and sequences' lengths and first own tiles."""
        most = WIDE // self.P * self.P
        ok = [0 <= n <= most for n in self.lens]
        lens = [int(n) if good and b not in skipped else 0
                for b, (n, good) in enumerate(zip(self.lens, ok))]
        prefix, start = [], [-1 if n == 0 else 0 for n in lens]
        for lo, hi in zip(self.group, self.group[1:]):
            # (a first sequence whose tree is bad lends its pages all the same)
            lead = next((b for b in range(lo, hi) if ok[b] and self.lens[b] - N >= TILE), None)
            share = {}
            for b in range(lo, hi):
                if lead is None or lens[b] == 0:
                    continue
                both = min(lens[b], int(self.lens[lead])) - N
                here = self.table[b, :max(0, both) // self.P + 1]
                differ = np.flatnonzero(here != self.table[lead, :len(here)])
                if len(differ):
                    both = min(both, differ[0] * self.P)
                if both >= TILE:
                    share[b] = both // TILE
            others = [x for b, x in share.items() if b != lead]
            prefix.append(min(others) if others else 0)
            for b in share:
                start[b] = prefix[-1]
        return prefix, lens, start

    def check(self, gpu_lib, N=1, skipped=(), **kw):
        (length, extra, first), status, outs = self.run(gpu_lib, N=N, **kw)
        prefix, lens, start = self.expect(N, skipped)
        G = len(self.group) - 1
        assert length[:G].tolist() == [TILE * x for x in prefix]
        assert extra[:G].tolist() == np.diff(self.group).tolist()
        assert length[G:].tolist() == lens and extra[G:].tolist() == start
        assert (first[:G] & 0xffff).tolist() == self.group[:-1]
        assert (first[G:] & 0xffff).tolist() == list(range(len(lens)))
        assert ((first[G:] >> 16) & 0xffff).tolist() == list(range(len(lens)))
        close(*outs)
        return status, prefix


def close(o, want, q, T):
    """Two results of the same sums in another order, each within its bound.  Keys and values are at
    most 1.5 in magnitude, so the sum of |q k| is at most 12 |q|; logits are fp32 sums of 64 products
    (64 * 2^-23 of that), which moves the result by twice as much of the largest value, 1.5;
    probabilities and the output are rounded to binary16 (2^-11 each; 2^-32 of the largest for
    small ones); fp32 sums over T positions add T * 2^-22."""
    d = 64 * 2.0 ** -23 * 12 * float(q.float().norm(dim=-1).max()) / 8 + 2.0 ** -20
    tol = 2 * 1.5 * (2 * d + 2 * 2.0 ** -11 + T * (2.0 ** -22 + 2.0 ** -32))
    assert float((o.float() - want.float()).abs().max()) <= tol


@pytest.mark.parametrize("groups, lens, P, N, lead", [
    ([(4, 10)], [700, 650, 641, 690], 64, 1, [5]),            # 640 tokens in common: all of them
    ([(4, 9)], [700, 650, 641, 690], 64, 1, [4]),             # 576: whole tiles of them
    ([(4, 10)], [700, 650, 641, 640], 64, 1, [4]),            # the last one's block lies in them
    ([(3, 1)], [300, 290, 280], 96, 1, [0]),                  # less than a tile
    ([(2, 4), (1, 3), (3, 2), (2, 0)], [129, 140, 500, 257, 256, 300, 400, 400], 128, 1,
     [1, 0, 1, 0]),
    ([(6, 8)], [600, 0, 520, 90, 7, 700], 64, 3, [4]),        # some hardly begun
    ([(5, 2)], [3500, 3400, 3329, 3600, 4000], 1664, 1, [26]),
])
def test_prefixes(gpu_lib, groups, lens, P, N, lead):
    s = Batch(np.random.default_rng(sum(lens)), groups, lens, P)
    status, prefix = s.check(gpu_lib, N)
    assert status == 0 and prefix == lead


@pytest.mark.parametrize("members", [9, 16, 17, 40, 130])
def test_large_groups(gpu_lib, members):
    """A group of a cluster of blocks: one of its sequences has the least in common."""
    rng = np.random.default_rng(members)
    s = Batch(rng, [(members, 6)], rng.integers(400, 500, members), 64)
    assert s.check(gpu_lib) == (0, [3])
    s.table[members - 2, 3] = s.table[members - 2, 6]     # another page: 192 tokens are left
    assert s.check(gpu_lib) == (0, [1])
    s.table[members // 2, 1] = s.table[members // 2, 6]   # none left: it does not count
    assert s.check(gpu_lib) == (0, [1])
    s.lens[0] = 100                                       # another sequence is the first
    assert s.check(gpu_lib) == (0, [1])


def test_a_cluster_with_sequences_that_are_skipped(gpu_lib):
    """Refused rows and bad trees in a group of a cluster, the first one among them."""
    rng = np.random.default_rng(1)
    s = Batch(rng, [(20, 6)], rng.integers(420, 500, 20), 64)
    parent = np.tile(np.array([-1, 0, 0], np.int32), (20, 1))
    for rows in ((0,), (0, 9, 19), (3, 4)):
        bad = parent.copy()
        bad[list(rows), 2] = 2
        status, prefix = s.check(gpu_lib, 3, skipped=rows, parent=bad)
        assert status == gpu_lib.GDN_ERR_BAD_TREE and prefix == [3]
        kept = s.lens.copy()
        s.lens[list(rows)] = -1
        status, prefix = s.check(gpu_lib, 3, parent=parent)
        assert status == gpu_lib.GDN_ERR_ROW_RANGE and prefix == [3]
        s.lens = kept


def test_a_cluster_and_sequences_of_no_group(gpu_lib):
    rng = np.random.default_rng(2)
    s = Batch(rng, [(40, 6)], rng.integers(400, 500, 40), 64)
    for group in ([7, 31], [0, 20], [20, 40], [13, 13], [1, 20, 39]):
        s.group = group
        status, prefix = s.check(gpu_lib)
        assert status == 0 and prefix == [3 * (b > a) for a, b in zip(group, group[1:])]


@pytest.mark.parametrize("group", [[0, 41], [-1, 40], [0, 30, 20, 40], [1 << 30, 1 << 30]])
def test_a_cluster_with_bad_offsets(gpu_lib, group):
    """Reported, and every sequence stands for itself."""
    rng = np.random.default_rng(3)
    s = Batch(rng, [(40, 6)], rng.integers(400, 500, 40), 64)
    s.group = group
    (length, extra, _), status, outs = s.run(gpu_lib)
    G = len(group) - 1
    assert status == gpu_lib.GDN_ERR_ROW_RANGE
    assert not length[:G].any() and not extra.any()
    assert np.array_equal(length[G:], s.lens)
    close(*outs)


@pytest.mark.parametrize("group_of, alone", [(699, 99), (4400, 0)])
def test_more_sequences_than_a_block_keeps(gpu_lib, group_of, alone):
    """One block, and each block of a cluster, with more than 512 sequences of its group, whose
    numbers wait in the workspace then."""
    rng = np.random.default_rng(group_of)
    s = Batch(rng, [(group_of, 2)] + [(1, 0)] * alone,
              rng.integers(260, 380, group_of + alone), 128)
    status, prefix = s.check(gpu_lib)
    assert status == 0 and prefix == [2] + [0] * alone
    row = group_of - 5
    s.table[row, 1] = s.table[row, 2]
    s.lens[3], s.lens[group_of - 1] = -1, 50
    status, prefix = s.check(gpu_lib)
    assert status == gpu_lib.GDN_ERR_ROW_RANGE and prefix == [1] + [0] * alone


def test_the_columns_that_the_lengths_need(gpu_lib):
    """A wide table's first columns, rows as far apart as before: short sequences are then read
    each for itself, with the full attention's bits."""
    t = torch()
    rng = np.random.default_rng(5)
    s = Batch(rng, [(4, 10)], [700, 650, 641, 690], 64)
    q = t.randn((4, 1, 6, 64), generator=t.Generator("cuda").manual_seed(1), device="cuda").half()
    ws = t.empty(gpu_lib.gdn_kv4_attention_shared_workspace_bytes(4, 1, 6, 1, 64, 1),
                 dtype=t.uint8, device="cuda")
    pages, table, lens, status = cuda(s.pages), i32(s.table), i32(s.lens), status_word()
    o, want = t.empty_like(q), t.empty_like(q)
    assert table[:, :11].stride(0) == table.shape[1] > 11
    kw = dict(scale=0.125, status=status)
    gpu_lib.gdn_kv4_attention_shared(q, pages, table[:, :11], lens, i32([0, 4]), o, ws, **kw)
    gpu_lib.gdn_kv4_attention(q, pages, table, lens, want, ws, **kw)
    assert int(status.item()) == 0 and t.equal(o, want)
