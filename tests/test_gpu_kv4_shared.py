"""Attention over the 4-bit cache for sequences that share pages, on the GPU against 64 bits, and
a run of branching, rotary append, both forms of the attention and commit together."""
import numpy as np
import pytest

import kv4_forms_reference as forms
import kv4_reference as ref
from gpu_helpers import torch
from test_gpu_kv4 import DT, cuda, i32, rand_trees, status_word, tdtype
from test_gpu_kv4_window import queries

pytestmark = pytest.mark.gpu


class Branches:
    """Sequences of several groups: the first shared[g] pages of a group's are the same ones.
    groups: (members, shared pages); lens: of all sequences.  The table is as wide as a
    million tokens, so that sharing pays by the sizes (narrow=True: no wider than
    needed, and each sequence is read for itself)."""

    def __init__(self, rng, groups, lens, H, D, P, narrow=False):
        self.H, self.D, self.P, self.lens = H, D, P, np.asarray(lens)
        held = [-(-max(0, n) // P) for n in lens]
        self.width = max(held) + 1 if narrow else -(-(1 << 20) // P)
        n_pages = sum(held) + 2
        order = list(rng.permutation(n_pages))
        self.table = np.full((len(lens), self.width), -1, np.int64)
        self.group, b = [0], 0
        for members, shared in groups:
            common = [order.pop() for _ in range(shared)]
            for _ in range(members):
                n = min(shared, held[b])
                self.table[b, :n] = common[:n]
                for j in range(n, held[b]):
                    self.table[b, j] = order.pop()
                b += 1
            self.group.append(b)
        self.pages = rng.integers(0, 256, (n_pages, H, P // 32, 36 * D), dtype=np.uint8)
        self.ks, self.vs = (rng.uniform(0.3, 2, H).astype(np.float32) for _ in range(2))
        self.cache = ref.Cache(self.pages, D)
        done = set()
        for b, n in enumerate(lens):
            for p in range(max(0, int(n))):
                at = (self.table[b, p // P], p % P)
                if at in done:
                    continue
                done.add(at)
                kc, ks = ref.quantise(rng.standard_normal((H, D)), self.ks)
                vc, vs = ref.quantise(rng.standard_normal((H, D)), self.vs)
                for h in range(H):
                    self.cache.put(at[0], h, at[1], kc[h], ks[h], vc[h], vs[h])

    def gpu(self):
        self.g_pages, self.g_table = cuda(self.pages), i32(self.table)
        self.g_len, self.g_ks, self.g_vs = i32(self.lens), cuda(self.ks), cuda(self.vs)
        self.g_group, self.status = i32(self.group), status_word()
        return dict(k_scale=self.g_ks, v_scale=self.g_vs, status=self.status)

    def space(self, gpu_lib, q, groups):
        t = torch()
        B, N, Hq, D = q.shape
        return t.full((gpu_lib.gdn_kv4_attention_shared_workspace_bytes(B, N, Hq, self.H, D,
                                                                       groups),),
                      255, dtype=t.uint8, device="cuda")

    def attend(self, gpu_lib, q, parent=None, ws=None):
        t = torch()
        kw = self.gpu()
        o = t.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
        lse = t.full(q.shape[:3], 5.0, device="cuda")
        ws = self.space(gpu_lib, q, len(self.group) - 1)
        par = None if parent is None else i32(parent)
        got = []
        for _ in range(2):   # the workspace as a call leaves it serves the next one: same bits
            gpu_lib.gdn_kv4_attention_shared(q, self.g_pages, self.g_table, self.g_len,
                                             self.g_group, o, ws, scale=q.shape[3] ** -0.5,
                                             parent=par, lse=lse, **kw)
            got.append((o.clone(), lse.clone()))
        assert t.equal(got[0][0], got[1][0]) and t.equal(got[0][1], got[1][1])
        return o, lse

    def attend_once(self, gpu_lib, q):
        t = torch()
        kw = self.gpu()
        o, lse = t.empty_like(q), t.empty(q.shape[:3], device="cuda")
        gpu_lib.gdn_kv4_attention_shared(q, self.g_pages, self.g_table, self.g_len, self.g_group,
                                         o, self.space(gpu_lib, q, len(self.group) - 1),
                                         scale=q.shape[3] ** -0.5, lse=lse, **kw)
        return o, lse

    def want(self, q, parent=None):
        N, D = q.shape[1], q.shape[3]
        return forms.attention(self.cache, self.table, self.lens, self.P, q.double().cpu().numpy(),
                               D ** -0.5, self.ks, self.vs, lambda b, n: forms.visible(
                                   n, N, None if parent is None else parent[b]))


CASES = [
    # dtype, groups (members, shared pages), lens, N, Hq, H, D, P, tree
    ("bf16", [(4, 10)], [700, 650, 641, 690], 1, 24, 4, 256, 64, False),
    ("bf16", [(2, 4)], [129, 140], 1, 1, 1, 64, 32, False),            # one shared tile
    ("f16", [(3, 9), (1, 5), (5, 7)], [600, 300, 290, 450, 230, 240, 250, 260, 700], 1, 8, 2, 128,
     32, False),
    ("bf16", [(4, 2)], [300, 200, 150, 400], 4, 6, 2, 64, 96, False),  # pages past whole tiles
    ("bf16", [(6, 8)], [600, 0, 520, 90, 7, 700], 3, 8, 2, 128, 64, False),  # some hardly begun
    ("f16", [(40, 6)], list(range(400, 440)), 1, 4, 1, 64, 64, False),  # more than a pass compares
    ("bf16", [(3, 4), (2, 3)], [600, 560, 580, 450, 420], 11, 24, 4, 256, 128, True),
    ("f16", [(8, 5)], [340, 341, 360, 352, 399, 330, 350, 345], 7, 16, 2, 128, 64, True),
    ("bf16", [(2, 0), (3, 4)], [300, 310, 280, 290, 300], 2, 4, 4, 64, 64, False),  # nothing shared
    ("bf16", [(5, 1)], [1700, 1800, 1690, 1900, 2000], 1, 16, 2, 256, 1664, False),
    ("f16", [(2, 5)], [500, 400], 22, 12, 2, 128, 64, False),          # 132 rows a sequence
    ("bf16", [(2, 4)], [300, 290], 16, 24, 4, 64, 64, False),          # rows that fill a tile
    ("bf16", [(3, 3)], [400, 300, 350], 1, 40, 1, 64, 128, False),     # 40 rows of a kv head
]


@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("dtype, groups, lens, N, Hq, H, D, P, tree", CASES)
def test_shared(gpu_lib, dtype, groups, lens, N, Hq, H, D, P, tree, narrow):
    rng = np.random.default_rng(sum(lens) + N * D + Hq)
    s = Branches(rng, groups, lens, H, D, P, narrow)
    parent = rand_trees(rng, len(lens), N) if tree else None
    q = queries(rng, len(lens), N, Hq, D, dtype)
    o, lse = s.attend(gpu_lib, q, parent)
    assert int(s.status.item()) == 0
    forms.check(o, lse, s.want(q, parent), max(lens), DT[dtype][1], D)


@pytest.mark.parametrize("group", [[0, 5], [1, 3], [0, 0, 2, 5], [2, 2], [0, 1, 2, 3, 4, 5],
                                   [3, 5]])
def test_any_groups_give_the_same_result(gpu_lib, group):
    """Groups with sequences that share nothing, empty ones, sequences outside of all groups."""
    rng = np.random.default_rng(40)
    s = Branches(rng, [(3, 5), (2, 3)], [400, 390, 350, 300, 290], 2, 64, 64)
    s.group = group
    q = queries(rng, 5, 2, 6, 64, "bf16")
    o, lse = s.attend(gpu_lib, q)
    assert int(s.status.item()) == 0
    forms.check(o, lse, s.want(q), 400, DT["bf16"][1], 64)


@pytest.mark.parametrize("group", [[0, 6], [-1, 5], [0, 4, 3, 5], [1 << 30, 1 << 30]])
def test_bad_groups_share_nothing_and_are_reported(gpu_lib, group):
    rng = np.random.default_rng(41)
    s = Branches(rng, [(5, 5)], [400, 390, 350, 380, 360], 2, 64, 64)
    s.group = group
    q = queries(rng, 5, 2, 6, 64, "bf16")
    o, lse = s.attend(gpu_lib, q)
    assert int(s.status.item()) == gpu_lib.GDN_ERR_ROW_RANGE
    forms.check(o, lse, s.want(q), 400, DT["bf16"][1], 64)


def test_skipped_sequences_leave_the_group_its_prefix(gpu_lib):
    """Lengths of -1 and 0 and a malformed tree give 0 and -infinity; the rest is as without."""
    rng, t = np.random.default_rng(42), torch()
    s = Branches(rng, [(6, 6)], [450, 430, 440, 420, 410, 400], 2, 128, 64)
    q = queries(rng, 6, 5, 4, 128, "bf16")
    parent = rand_trees(rng, 6, 5)
    for row, n, code in ((0, -1, gpu_lib.GDN_ERR_ROW_RANGE), (2, 0, 0),
                         (3, 1 << 21, gpu_lib.GDN_ERR_ROW_RANGE),
                         (4, None, gpu_lib.GDN_ERR_BAD_TREE)):
        lens, par = s.lens.copy(), parent.copy()
        if n is None:
            par[row, 2] = 2
        else:
            s.lens[row] = n
        o, lse = s.attend(gpu_lib, q, par)
        assert int(s.status.item()) == code
        assert not o[row].any() and t.isinf(lse[row]).all()
        s.lens = lens.copy()
        s.lens[row] = 0
        forms.check(o, lse, s.want(q, parent), 450, DT["bf16"][1], 128)
        s.lens = lens


def test_bad_pages_are_left_out_and_reported(gpu_lib):
    """A bad page number in the shared part, and one in a sequence's own."""
    rng = np.random.default_rng(43)
    for row, entry in ((None, 2), (1, 7)):
        s = Branches(rng, [(3, 6)], [450, 500, 420], 2, 64, 64)
        rows = slice(None) if row is None else row
        q = queries(rng, 3, 2, 6, 64, "f16")
        good = s.table.copy()
        s.table[rows, entry] = 1 << 20
        o, lse = s.attend(gpu_lib, q)
        assert int(s.status.item()) == gpu_lib.GDN_ERR_PAGE_RANGE

        def seen(b, n):
            x = forms.visible(n, 2)
            if row is None or b == row:
                x[:, entry * 64:entry * 64 + 64] = False
            return x
        want = forms.attention(s.cache, good, s.lens, 64, q.double().cpu().numpy(), 64 ** -0.5,
                               s.ks, s.vs, seen)
        forms.check(o, lse, want, 500, DT["f16"][1], 64)


def test_pages_copied_on_write_are_not_shared(gpu_lib):
    """The last common page of some has other contents (a copy that was written): what is shared
    ends before it, and each sequence reads its own."""
    rng = np.random.default_rng(44)
    s = Branches(rng, [(4, 6)], [384, 384, 384, 384], 1, 64, 64)
    spare = s.pages.shape[0]
    s.pages = np.concatenate((s.pages, s.pages[s.table[2, 3:4]], s.pages[s.table[0, 5:6]]))
    s.cache = ref.Cache(s.pages, 64)
    s.table[2, 3], s.table[0, 5] = spare, spare + 1      # entries 3 and 5 of two rows
    for row, p in ((2, 200), (0, 330)):
        kc, ks = ref.quantise(rng.standard_normal((1, 64)), s.ks)
        vc, vs = ref.quantise(5 * rng.standard_normal((1, 64)), s.vs)
        s.cache.put(s.table[row, p // 64], 0, p % 64, kc[0], ks[0], vc[0], vs[0])
    q = queries(rng, 4, 1, 6, 64, "bf16")
    o, lse = s.attend(gpu_lib, q)
    forms.check(o, lse, s.want(q), 384, DT["bf16"][1], 64)


def test_large_logits_on_either_side(gpu_lib):
    """All the weight in the shared part, or all in the own one, with logits far apart."""
    rng = np.random.default_rng(45)
    s = Branches(rng, [(4, 4)], [300, 310, 290, 280], 1, 64, 64)
    q = queries(rng, 4, 1, 4, 64, "bf16")
    q *= 8
    for p, row in ((100, 0), (270, 1)):
        kc, ks = ref.quantise(3 * q[row, 0, :1].double().cpu().numpy(), s.ks)
        vc, vs = ref.quantise(np.full((1, 64), 2.0), s.vs)
        s.cache.put(s.table[row, p // 64], 0, p % 64, kc[0], ks[0], vc[0], vs[0])
    o, lse = s.attend(gpu_lib, q)
    want = s.want(q)
    assert want[1].max() - want[1].min() > 50
    forms.check(o, lse, want, 310, DT["bf16"][1], 64)


def test_many_sequences(gpu_lib):
    """More sequences, and more groups, than a block keeps the numbers of."""
    rng = np.random.default_rng(46)
    B = 1300
    lens = rng.integers(128, 160, B)
    s = Branches(rng, [(2, 4)] * 600 + [(100, 4)], lens, 1, 64, 32, narrow=True)
    q = queries(rng, B, 1, 2, 64, "f16")
    o, lse = s.attend(gpu_lib, q)
    assert int(s.status.item()) == 0
    forms.check(o, lse, s.want(q), 160, DT["f16"][1], 64)


def test_two_graphs_with_workspaces_of_their_own(gpu_lib):
    """Two captured calls replayed on two streams at once, lengths and groups rewritten."""
    rng, t = np.random.default_rng(47), torch()
    runs = []
    for k in range(2):
        s = Branches(rng, [(3, 6), (3, 5)], [500, 480, 450, 400, 390, 380], 2, 128, 64)
        kw = s.gpu()
        q = queries(rng, 6, 2, 4, 128, "bf16")
        o = t.empty(q.shape, dtype=q.dtype, device="cuda")
        stream = t.cuda.Stream()
        stream.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(stream):
            call = gpu_lib.bind_kv4_attention_shared(q, s.g_pages, s.g_table, s.g_len, s.g_group, o,
                                                     s.space(gpu_lib, q, 2), scale=128 ** -0.5,
                                                     **kw)
            call()
            stream.synchronize()
            g = t.cuda.CUDAGraph()
            with t.cuda.graph(g, stream=stream):
                call()
        runs.append((s, q, o, g, stream, call))
    for step in range(3):
        for s, *_ in runs:
            s.lens = s.lens - 30 * (step > 0)
            s.group = [[0, 3, 6], [0, 2, 5], [1, 1, 6]][step]
            s.g_len.copy_(i32(s.lens))
            s.g_group.copy_(i32(s.group))
        t.cuda.synchronize()
        for _ in range(3):
            for s, q, o, g, stream, _c in runs:
                with t.cuda.stream(stream):
                    g.replay()
        t.cuda.synchronize()
        for s, q, o, *_ in runs:
            assert int(s.status.item()) == 0
            forms.check(o, None, s.want(q), 500, DT["bf16"][1], 128)


def test_a_large_group_in_a_graph(gpu_lib):
    """One group of more sequences than a block of the plan takes, captured; replays follow the
    table, and the bits are those of the call itself."""
    rng, t = np.random.default_rng(49), torch()
    s = Branches(rng, [(20, 6)], rng.integers(400, 480, 20), 1, 64, 64)
    kw = s.gpu()
    q = queries(rng, 20, 1, 4, 64, "f16")
    o = t.empty(q.shape, dtype=q.dtype, device="cuda")
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        call = gpu_lib.bind_kv4_attention_shared(q, s.g_pages, s.g_table, s.g_len, s.g_group, o,
                                                 s.space(gpu_lib, q, 1), scale=0.125, **kw)
        call()
        side.synchronize()
        first = o.clone()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            call()
    for step in range(2):
        if step:   # one row's third page becomes a page of its own, of the same contents
            s.g_pages = None
            spare = s.table[7, 6]
            s.table[7, 2], s.lens[7] = spare, 300
            s.pages[spare] = s.pages[s.table[0, 2]]
            call._keep[2].copy_(cuda(s.pages))
            s.g_table.copy_(i32(s.table))
            s.g_len.copy_(i32(s.lens))
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        assert int(s.status.item()) == 0
        assert step or t.equal(o, first)
        forms.check(o, None, s.want(q), 480, DT["f16"][1], 64)


def test_lengths_written_just_before_the_call(gpu_lib):
    """Lengths and tables rewritten on the stream between calls that follow each other: every call
    goes by what they are then."""
    rng, t = np.random.default_rng(50), torch()
    s = Branches(rng, [(4, 5), (3, 4)], [500, 480, 450, 470, 400, 390, 380], 2, 64, 64)
    kw = s.gpu()
    q = queries(rng, 7, 2, 4, 64, "bf16")
    ws = [s.space(gpu_lib, q, 2), t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(7, 2, 4, 2, 64),
                                          dtype=t.uint8, device="cuda")]
    lens = [i32(s.lens - d) for d in (0, 130, 64, 250, 1, 300)]

    def run(out, k):
        if k % 2:
            gpu_lib.gdn_kv4_attention_window(q, s.g_pages, s.g_table, s.g_len, out, ws[1],
                                             scale=0.125, window=150, sinks=3, **kw)
        else:
            gpu_lib.gdn_kv4_attention_shared(q, s.g_pages, s.g_table, s.g_len, s.g_group, out,
                                             ws[0], scale=0.125, **kw)

    alone = []
    for n in lens:
        for k in range(2):
            s.g_len.copy_(n)
            t.cuda.synchronize()
            alone.append(t.empty(q.shape, dtype=q.dtype, device="cuda"))
            run(alone[-1], k)
            t.cuda.synchronize()
    for order in ((0, 1, 2, 3, 4, 5), (5, 3, 1, 0, 2, 4)):
        outs = [t.empty(q.shape, dtype=q.dtype, device="cuda") for _ in alone]
        for i in order:
            for k in range(2):
                t.add(lens[i], 0, out=s.g_len)
                run(outs[2 * i + k], k)
        t.cuda.synchronize()
        for got, want in zip(outs, alone):
            assert t.equal(got, want)
    assert int(s.status.item()) == 0


def test_a_nan_query_stays_with_its_rows(gpu_lib):
    """A NaN and an infinity in one branch's queries: its rows are no numbers, the others' stay
    within their bound."""
    rng, t = np.random.default_rng(51), torch()
    s = Branches(rng, [(5, 5)], [500, 480, 450, 470, 400], 2, 128, 64)
    q = queries(rng, 5, 3, 4, 128, "bf16").contiguous()
    want = s.want(q)
    q[1, 2, 3, 5], q[3, 0, 0, 9] = float("nan"), float("inf")
    o, lse = s.attend_once(gpu_lib, q)
    bad = [(1, 2, 3), (3, 0, 0)]
    for at in bad:
        assert t.isnan(o[at]).any()
        o[at], lse[at] = t.from_numpy(want[0][at]).to(o.dtype), float(want[1][at])
    forms.check(o, lse, want, 500, DT["bf16"][1], 128)


def test_rounds_of_branches(gpu_lib):
    """A prompt branched three ways; two rounds of reserve, rotary append, attention (over shared
    pages, and through a window), commit and release without the host, against the reference.
    The second round finds no page for one branch."""
    rng, t = np.random.default_rng(48), torch()
    H, Hq, D, P, N, F, prompt = 2, 6, 64, 32, 5, 3, 170
    n_pages = 12
    pages = t.zeros(n_pages, H, 1, 36 * D, dtype=t.uint8, device="cuda")
    table, kv_len = i32(np.full((F + 1, 32768), -1)), i32(np.zeros(F + 1))
    holders, status = i32(np.zeros(n_pages)), status_word()
    ws = t.empty(max(gpu_lib.gdn_kv4_reserve_workspace_bytes(F),
                     gpu_lib.gdn_kv4_attention_workspace_bytes(F, N, Hq, H, D),
                     gpu_lib.gdn_kv4_attention_shared_workspace_bytes(F, N, Hq, H, D, 1)),
                 dtype=t.uint8, device="cuda")
    a = np.arange(400)[:, None] * 10.0 ** (-np.arange(16) / 4)
    cs = np.stack((np.cos(a), np.sin(a)), 1).astype(np.float32)
    g_cs = cuda(cs)
    pool = (table, kv_len, holders)

    def projections(B, n):
        return [t.from_numpy(rng.standard_normal((B, n, h, D))).cuda().to(t.bfloat16)
                for h in (Hq, H, H)]

    # the prompt, in row 0
    q, k, v = projections(1, prompt)
    gpu_lib.gdn_kv4_reserve(pages, *pool, i32([0]), i32([prompt]), ws, status=status)
    pos = np.arange(prompt)[None, None]
    out = t.empty_like(q)
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), g_cs, pages, table[:1], kv_len[:1], out,
                                  status=status)
    # what each branch's sequence holds: turned keys, values
    told = [forms.turned(k.float().cpu().numpy(), pos, cs, None, False)[0], v.float().cpu().numpy()[0]]
    hold = [list(told) for _ in range(F)]
    rows, group = i32(np.arange(1, F + 1)), i32([0, F])
    gpu_lib.gdn_kv4_fork(*pool, i32([0] * F), rows, page_tokens=P, status=status)
    gpu_lib.gdn_kv4_release(*pool, i32([0]), i32([0]), page_tokens=P, status=status)
    granted, committed = i32([0] * F), i32([0] * F)
    lens = np.array([prompt] * F)
    for step in range(2):
        parent = rand_trees(rng, F, N)
        depth = np.array([[len(ref.path_of(p, n)) - 1 for n in range(N)] for p in parent])
        q, k, v = projections(F, N)
        block = kv_len[1:] + N
        if step == 1:       # the last branch asks for more than there is
            block = block + i32([0, 0, 150])
        gpu_lib.gdn_kv4_reserve(pages, *pool, rows, block, ws, granted=granted, status=status)
        served = (granted > 0).tolist()
        assert served == [True, True, step == 0]
        pos = lens[:, None] + depth
        q_out = t.empty_like(q)
        gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos[None]), g_cs, pages, table[1:], granted,
                                      q_out, status=status)
        o, lse = t.empty_like(q), t.empty(F, N, Hq, device="cuda")
        ow, lw = t.empty_like(o), t.empty_like(lse)
        par = i32(parent)
        gpu_lib.gdn_kv4_attention_shared(q_out, pages, table[1:], granted, group, o, ws, scale=0.2,
                                         parent=par, lse=lse, status=status)
        gpu_lib.gdn_kv4_attention_window(q_out, pages, table[1:], granted, ow, ws, scale=0.2,
                                         window=40, sinks=4, parent=par, lse=lw, status=status)
        accept = np.array([N - 1, 2, 1])
        gpu_lib.gdn_kv4_commit(pages, table[1:], granted, i32(accept), committed, N=N, parent=par,
                               status=status)
        gpu_lib.gdn_kv4_release(*pool, rows, committed, page_tokens=P, status=status)
        # the reference: one cache a branch, quantised from what it was told
        want_q = t.from_numpy(forms.turned(q.float().cpu().numpy(), pos[None], cs, None,
                                           False)).to(t.bfloat16)
        kt, vt = forms.turned(k.float().cpu().numpy(), pos[None], cs, None, False), v.float().cpu().numpy()
        ones = np.ones(H, np.float32)
        for b in range(F):
            if not served[b]:
                assert not q_out[b].any() and not o[b].any() and not ow[b].any()
                assert t.isinf(lse[b]).all()
                continue
            assert t.equal(q_out[b].cpu(), want_q[b])
            keys, vals = (np.concatenate((hold[b][i], (kt, vt)[i][b])) for i in (0, 1))
            L = len(keys)
            cache = ref.Cache(np.zeros((L // P + 1, H, 1, 36 * D), np.uint8), D)
            own = np.arange(L // P + 1)[None]
            ref.append(cache, own, [L], P, keys[None], vals[None], ones, ones)
            for got, glse, window, sinks in ((o, lse, None, 0), (ow, lw, 40, 4)):
                want = forms.attention(cache, own, [L], P, want_q[b:b + 1].double().numpy(), 0.2,
                                       ones, ones, lambda _, n: forms.visible(n, N, parent[b],
                                                                              window, sinks))
                forms.check(got[b:b + 1], glse[b:b + 1], want, L, DT["bf16"][1], D)
            path = ref.path_of(parent[b], accept[b])
            hold[b] = [np.concatenate((hold[b][i], (kt, vt)[i][b][path])) for i in (0, 1)]
            lens[b] += len(path)
        assert kv_len[1:].tolist() == lens.tolist()
    assert int(status.item()) == gpu_lib.GDN_ERR_POOL_EMPTY
