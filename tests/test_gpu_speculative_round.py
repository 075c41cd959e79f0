"""The example's speculative rounds on the GPU: after every commit the caches hold
exactly what the accepted tokens alone would have left there."""
import os
import sys

import pytest

from gpu_helpers import torch
from kv4_reference import path_of

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


def test_example_runs(example, capsys):
    example.main(rounds=2, B=2, prompt=70)
    assert "round 1" in capsys.readouterr().out


def test_rounds_equal_the_accepted_tokens_alone(example, gpu_lib):
    t, gdn = torch(), gpu_lib
    B, N, prompt = 3, 22, 45
    m = example.Mixers(B, N=N, recurrent=1)
    _, _, _, Hq, Hkv, D = m.shape
    m.prompt(prompt)
    kept_k, kept_v = (t.empty(B, prompt, Hkv, D, device="cuda") for _ in range(2))
    gdn.gdn_kv4_read(m.pages, m.table, m.length, kept_k, kept_v)
    want = [(kept_k[b], kept_v[b]) for b in range(B)]
    host = t.Generator().manual_seed(5)
    for _ in range(4):
        parent = example.random_trees(B, N, host)
        accept = t.randint(N, (B,), generator=host, dtype=t.int32)
        qkv = m.normal(B, N, (Hq + 2 * Hkv) * D, dtype=t.bfloat16)
        o, _ = m.verify(parent.cuda(), qkv, [example.recurrent_inputs(m)])
        # what the block left in the cache, node by node
        k, v = (t.empty(B, N, Hkv, D, device="cuda") for _ in range(2))
        gdn.gdn_kv4_read(m.pages, m.table, m.length, k, v)
        # the accepted node's output is that of a chain of its path (float64)
        for b in range(B):
            path = path_of(parent[b].tolist(), int(accept[b]))
            want[b] = tuple(t.cat((w, x[b, path])) for w, x in zip(want[b], (k, v)))
            q = qkv[b, path[-1], :Hq * D].view(Hq, D).double()
            kk, vv = (x.double().repeat_interleave(Hq // Hkv, 1) for x in want[b])
            p = t.softmax(t.einsum("hd,nhd->hn", q, kk) * D ** -0.5, -1)
            ref = t.einsum("hn,nhd->hd", p, vv)
            weight = t.einsum("hn,nhd->hd", p, vv.abs())
            # bf16 output, binary16 probabilities, fp32 logits (D * 2^-23 of a logit below 64)
            tol = 2.0 ** -8 * ref.abs() + weight * (2.0 ** -11 + 2 * 64 * D * 2.0 ** -23)
            assert bool(((o[b, path[-1]].double() - ref).abs() <= tol).all())
        m.commit(parent.cuda(), accept.cuda())
        lengths = m.length.tolist()
        assert lengths == [w[0].shape[0] for w in want]
        longest = max(lengths)
        k, v = (t.empty(B, longest, Hkv, D, device="cuda") for _ in range(2))
        gdn.gdn_kv4_read(m.pages, m.table, m.length, k, v)
        for b, n in enumerate(lengths):
            assert t.equal(k[b, longest - n:], want[b][0])
            assert t.equal(v[b, longest - n:], want[b][1])
        held = int((m.ref > 0).sum())
        assert held == sum(-(-n // m.page_tokens) for n in lengths)
    assert int(m.status.item()) == 0


def test_branches_share_pages_until_they_write(example, gpu_lib):
    """Two branches of one sequence append different tokens: each sees its own, the
    source keeps its page."""
    t, gdn = torch(), gpu_lib
    i32 = dict(dtype=t.int32, device="cuda")
    H, D, P = 2, 128, 64
    pages = t.zeros(12, H, P // 32, 36 * D, dtype=t.uint8, device="cuda")
    table, length = t.full((3, 4), -1, **i32), t.zeros(3, **i32)
    ref, status = t.zeros(12, **i32), t.zeros(1, **i32)
    ws = t.empty(gdn.gdn_kv4_reserve_workspace_bytes(2), dtype=t.uint8, device="cuda")
    pool = (table, length, ref)
    gen = t.Generator(device="cuda").manual_seed(2)
    k0 = t.randn(1, 100, H, D, generator=gen, device="cuda")
    gdn.gdn_kv4_reserve(pages, *pool, t.tensor([0], **i32), t.tensor([100], **i32), ws,
                        status=status)
    gdn.gdn_kv4_append(k0, -k0, pages, table[:1], length[:1], status=status)
    both = t.tensor([1, 2], **i32)
    gdn.gdn_kv4_fork(*pool, t.tensor([0, 0], **i32), both, page_tokens=P, status=status)
    assert ref.sum().item() == 6 and (ref > 0).sum().item() == 2
    gdn.gdn_kv4_reserve(pages, *pool, both, t.tensor([103, 130], **i32), ws, status=status)
    new = [t.randn(1, n, H, D, generator=gen, device="cuda") for n in (3, 30)]
    for row, x in zip((1, 2), new):
        gdn.gdn_kv4_append(x, -x, pages, table[row:row + 1], length[row:row + 1], status=status)
    read = {}
    for row, n in ((0, 100), (1, 103), (2, 130)):
        k, v = (t.empty(1, n, H, D, device="cuda") for _ in range(2))
        gdn.gdn_kv4_read(pages, table[row:row + 1], length[row:row + 1], k, v, status=status)
        assert t.equal(k, -v)
        read[row] = k[0]
    assert t.equal(read[1][:100], read[0]) and t.equal(read[2][:100], read[0])
    lone_pages = t.zeros_like(pages)
    for row, x in zip((1, 2), new):   # the appended tokens as a cache of their own holds them
        n = x.shape[1]
        k, v = t.empty_like(x), t.empty_like(x)
        one = t.tensor([n], **i32)
        tab = t.tensor([[row]], **i32)
        gdn.gdn_kv4_append(x, -x, lone_pages, tab, one, status=status)
        gdn.gdn_kv4_read(lone_pages, tab, one, k, v, status=status)
        assert t.equal(read[row][100:], k[0])
    # each branch has a page of its own for the shared page's tail
    assert int(table[1, 1]) != int(table[0, 1]) != int(table[2, 1])
    gdn.gdn_kv4_release(*pool, t.tensor([0, 1, 2], **i32), t.tensor([0, 0, 0], **i32),
                        page_tokens=P, status=status)
    assert not ref.any() and int(status.item()) == 0
