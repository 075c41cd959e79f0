"""One speculative round of a hybrid model's sequence mixers, on the GPU.

Three recurrent layers and one full-attention layer verify a draft tree and
commit its accepted path:

  recurrent layer   gdn_verify_tree over the block, every node's state persisted;
                    gdn_commit_accepted puts the accepted node's state in the cache
  attention layer   gdn_kv4_reserve makes room and says for which sequences it
                    could, gdn_kv4_append quantises the block's keys and values
                    into the 4-bit cache,
                    gdn_kv4_attention attends under the ancestor mask;
                    gdn_kv4_commit moves the accepted path together and
                    gdn_kv4_release gives the pages past it back

The projections around the mixers are random tensors here.  Nothing in a round
waits for the host: lengths, tables and page counts are device memory.  A sequence
that finds no page sits the round out: its granted length is -1, so no call touches
its tokens, and no node of it is accepted in any layer.

    python examples/speculative_round.py
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import hybrid_gated_deltanet_delta_gb300 as gdn  # noqa: E402


class Mixers:
    """State and caches of `recurrent` recurrent layers and one attention layer."""

    def __init__(self, B, *, recurrent=3, Hk=4, Hv=12, d=128, Hq=24, Hkv=4, D=256, N=22,
                 page_tokens=64, max_tokens=1024, seed=0):
        self.B, self.N, self.shape = B, N, (Hk, Hv, d, Hq, Hkv, D)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        new = dict(device="cuda")
        self.state = [0.05 * self.normal(B, Hv, d, d) for _ in range(recurrent)]
        self.snap = torch.empty(B, N, Hv, d, d, **new)
        width = -(-(max_tokens + N) // page_tokens)
        n_pages = B * width
        self.page_tokens = page_tokens
        self.pages = torch.empty(n_pages, Hkv, page_tokens // 32, 36 * D, dtype=torch.uint8, **new)
        i32 = dict(dtype=torch.int32, **new)
        self.table = torch.full((B, width), -1, **i32)
        self.length = torch.zeros(B, **i32)        # tokens committed
        self.ref = torch.zeros(n_pages, **i32)
        self.rows = torch.arange(B, **i32)
        self.status = torch.zeros(1, **i32)
        self.committed = torch.zeros(B, **i32)
        self.block = torch.zeros(B, **i32)         # tokens with the block; -1: no page for it
        self.reserve_ws = torch.empty(gdn.gdn_kv4_reserve_workspace_bytes(B), dtype=torch.uint8,
                                      **new)

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.gen, device="cuda").to(dtype)

    def _append(self, k, v, grown):
        """Room for the block, then its keys and values at its end."""
        gdn.gdn_kv4_reserve(self.pages, self.table, self.length, self.ref, self.rows, grown,
                            self.reserve_ws, granted=self.block, status=self.status)
        gdn.gdn_kv4_append(k, v, self.pages, self.table, self.block, status=self.status)

    def prompt(self, tokens):
        """A prompt of the same number of tokens for every sequence (attention layer)."""
        _, _, _, Hq, Hkv, D = self.shape
        qkv = self.normal(self.B, tokens, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
        self._append(k, v, self.length + tokens)
        return self._attend(q, None)

    def _attend(self, q, parent):
        B, N, Hq, D = q.shape
        Hkv = self.shape[4]
        ws = torch.empty(gdn.gdn_kv4_attention_workspace_bytes(B, N, Hq, Hkv, D),
                         dtype=torch.uint8, device="cuda")
        o = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        gdn.gdn_kv4_attention(q, self.pages, self.table, self.block, o, ws, scale=D ** -0.5,
                              parent=parent, status=self.status)
        return o

    def verify(self, parent, qkv, recurrent_inputs):
        """Verify one tree a sequence.  qkv [B,N,(Hq+2*Hkv)*D] of the attention
        layer; recurrent_inputs: q, k, v, alpha, beta of each recurrent layer."""
        _, _, _, Hq, Hkv, D = self.shape
        self.blocks = []
        for state, x in zip(self.state, recurrent_inputs):
            snap = torch.empty_like(self.snap)
            o = torch.empty(x[2].shape, device="cuda")
            gdn.gdn_verify_tree(*x, state, snap, o, parent, status=self.status)
            self.blocks.append((snap, o))
        q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
        self._append(k, v, self.length + self.N)
        return self._attend(q, parent), [o for _, o in self.blocks]

    def commit(self, parent, accept):
        """Commit the path to accept[b] of every sequence's tree, in every layer."""
        _, Hv, d = self.shape[:3]
        accept = torch.where(self.block < 0, -1, accept)
        for state, (snap, _) in zip(self.state, self.blocks):
            gdn.gdn_commit_accepted(snap, accept, state, B=self.B, N=self.N, Hv=Hv, dk=d, dv=d,
                                    status=self.status)
        gdn.gdn_kv4_commit(self.pages, self.table, self.block, accept, self.committed, N=self.N,
                           parent=parent, status=self.status)
        gdn.gdn_kv4_release(self.table, self.length, self.ref, self.rows, self.committed,
                            page_tokens=self.page_tokens, status=self.status)


def random_trees(B, N, gen, max_depth=16):
    """parent [B,N] of random trees, parents before children."""
    parent = torch.full((B, N), -1, dtype=torch.int32)
    for b in range(B):
        depth = [1]
        for n in range(1, N):
            open_nodes = [i for i in range(n) if depth[i] < max_depth]
            p = open_nodes[int(torch.randint(len(open_nodes), (1,), generator=gen))]
            parent[b, n] = p
            depth.append(depth[p] + 1)
    return parent


def recurrent_inputs(m):
    """Random inputs of one recurrent layer's block: unit q and k, gates in (0, 1)."""
    Hk, Hv, d = m.shape[:3]
    q, k = (torch.nn.functional.normalize(m.normal(m.B, m.N, Hk, d), dim=-1).to(torch.bfloat16)
            for _ in range(2))
    v = m.normal(m.B, m.N, Hv, d, dtype=torch.bfloat16)
    alpha = 0.9 + 0.1 * torch.sigmoid(m.normal(m.B, m.N, Hv))
    beta = torch.sigmoid(m.normal(m.B, m.N, Hv))
    return q, k, v, alpha, beta


def main(rounds=4, B=4, prompt=300):
    m = Mixers(B)
    m.prompt(prompt)
    host = torch.Generator().manual_seed(1)
    for step in range(rounds):
        parent = random_trees(B, m.N, host).cuda()
        accept = torch.randint(m.N, (B,), generator=host, dtype=torch.int32).cuda()
        _, _, _, Hq, Hkv, D = m.shape
        qkv = m.normal(B, m.N, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16)
        o, outs = m.verify(parent, qkv, [recurrent_inputs(m) for _ in m.state])
        m.commit(parent, accept)
        print(f"round {step}: attention output rms {o.float().square().mean().sqrt():.3f}, "
              f"recurrent {outs[0].square().mean().sqrt():.3f}, lengths {m.length.tolist()}, "
              f"pages held {int((m.ref > 0).sum())}")
    code = int(m.status.item())
    if code:
        raise SystemExit(gdn.status_string(code))


if __name__ == "__main__":
    main()
