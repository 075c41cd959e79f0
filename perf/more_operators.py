"""Timed cases of what stands around the 4-bit key/value cache's append and attention.

  rotate   gdn_kv4_append_rotary of a block (or a whole prompt): queries and keys
           rotated by their positions on one or three axes (text; time, height and
           width of images and video), the queries out, the keys and values
           quantised into the cache; and gdn_kv4_read of what it then holds
  window   gdn_kv4_attention_window: the block's queries over the first few tokens
           and the last ones of their path
  shared   gdn_kv4_attention_shared: the queries of sequences that were branched
           from common prompts and still hold the same pages for them

`run` is the plain form (elementary torch operations in 32 bits) unless `own`
is set, in which case it makes the framework's calls.

A stored value is e2m1 code x e4m3 scale (16 channels of one token) x a scale
per head; 32 tokens of one head make a record of 36*D bytes: K codes
[D/32][32 tokens][16], V codes [D][16], K scales [32][D/16], V scales [D/16][32].
"""
import math
import random

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
HEADS = ((24, 4, 256), (32, 8, 128), (16, 4, 64), (8, 8, 128), (16, 2, 256), (12, 4, 128))
BASE = 10000.0       # of the rotation's frequencies


def listed():
    return [
        # one decoded token of text: the call's latency
        dict(name="rotate_one", op="rotate", B=1, N=1, Hq=24, Hkv=4, D=256, page=64, longest=700,
             shortest=700, pairs=32, axes=3, adjacent=False, dtype="bf16"),
        # a verification block of eight sequences
        dict(name="rotate_chain16x8", op="rotate", B=8, N=16, Hq=24, Hkv=4, D=256, page=64,
             longest=4096, shortest=1001, pairs=32, axes=3, adjacent=False, dtype="bf16"),
        # a decode batch whose heads are rotated whole, pairs of neighbouring channels
        dict(name="rotate_batch48", op="rotate", B=48, N=1, Hq=32, Hkv=8, D=128, page=32,
             longest=8192, shortest=0, pairs=64, axes=1, adjacent=True, dtype="f16"),
        # a whole prompt of text and an image
        dict(name="rotate_prompt8192", op="rotate", B=1, N=8192, Hq=24, Hkv=4, D=256, page=64,
             longest=8192, shortest=8192, pairs=32, axes=3, adjacent=False, dtype="bf16"),
        # one sequence decoding at 128K tokens through a window of 4,096 and four sinks
        dict(name="window_one_131072", op="window", B=1, N=1, Hq=24, Hkv=4, D=256, page=1664,
             longest=131072, shortest=131072, window=4096, sinks=4, tree=False, dtype="bf16"),
        # a full decode batch of uneven sequences, some shorter than the window
        dict(name="window_batch48", op="window", B=48, N=1, Hq=32, Hkv=8, D=128, page=32,
             longest=8192, shortest=0, window=1024, sinks=4, tree=False, dtype="f16"),
        # draft trees of a batch, verified through a window that ends inside a tile
        dict(name="window_tree22x8", op="window", B=8, N=22, Hq=24, Hkv=4, D=256, page=64,
             longest=16384, shortest=12001, window=2047, sinks=64, tree=True, dtype="bf16"),
        # one 2,048-token piece of a long prompt
        dict(name="window_prompt2048", op="window", B=1, N=2048, Hq=24, Hkv=4, D=256, page=64,
             longest=8192, shortest=8192, window=1024, sinks=128, tree=False, dtype="bf16"),
        # four answers to one short question, a token each: the call's latency
        dict(name="shared_4x700", op="shared", B=4, groups=1, N=1, Hq=24, Hkv=4, D=256, page=64,
             prefix=640, longest=700, shortest=650, tree=False, dtype="bf16"),
        # 32 answers sampled from one prompt of 32K tokens
        dict(name="shared_32x32768", op="shared", B=32, groups=1, N=1, Hq=24, Hkv=4, D=256,
             page=64, prefix=32768, longest=33768, shortest=32800, tree=False, dtype="bf16"),
        # eight prompts branched eight ways each, draft chains of four
        dict(name="shared_8x8_chain4", op="shared", B=64, groups=8, N=4, Hq=32, Hkv=8, D=128,
             page=32, prefix=4096, longest=5000, shortest=4200, tree=False, dtype="f16"),
        # two prompts of 16K branched eight ways each, draft trees of eleven nodes
        dict(name="shared_2x8_tree11", op="shared", B=16, groups=2, N=11, Hq=24, Hkv=4, D=256,
             page=128, prefix=16384, longest=17000, shortest=16500, tree=True, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hq, Hkv, D = rng.choice(HEADS)
    page = rng.choice((32, 64, 96, 128, 1664))
    op = rng.choice(("rotate", "window", "shared"))
    if op == "rotate":
        N = rng.choice((1, rng.randint(2, 64), _spread(rng, 65, 8192)))
        B = _spread(rng, 1, 64) if N <= 64 else 1
        longest = N + _spread(rng, 1, 4096)
        if N > 64:
            longest = max(N, min(longest, 8192))
        axes, dtype = rng.choice((1, 3)), rng.choice(("bf16", "f16", "f32"))
        if dtype == "f32" and N > 4096:
            N //= 2
        return dict(op=op, B=B, N=N, Hq=min(Hq, 24), Hkv=min(Hkv, 4), D=D, page=page,
                    longest=longest, shortest=rng.randint(0 if N <= 64 else N, longest),
                    pairs=rng.choice((8, 16, 24, 32, D // 4, D // 2)), axes=axes,
                    adjacent=rng.random() < 0.4, dtype=dtype)
    if op == "window":
        N = rng.choice((1, 1, rng.randint(2, 22), rng.randint(2, 64), _spread(rng, 65, 2048)))
        B = 1 if N > 64 else _spread(rng, 1, 48)
        longest = max(N + 1, _spread(rng, 40, min(131072, (1 << 27) // (B * Hkv * D))))
        while B * N * Hq * D * longest > 8e10:
            longest //= 2
        longest = max(longest, N + 1)
        window = _spread(rng, 1, 4096)
        while window > 1 and B * N * Hq * D * (window + 300) > 1.4e10:  # the listed prompt's work
            window //= 2
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, page=page, longest=longest,
                    shortest=rng.randint(0 if N <= 64 else N, longest), window=window,
                    sinks=rng.choice((0, 1, 4, rng.randint(5, 300))),
                    tree=N <= 64 and rng.random() < 0.4, dtype=rng.choice(("bf16", "f16")))
    groups, members = _spread(rng, 1, 8), _spread(rng, 1, 32)
    while groups * members > 64:
        members = max(1, members // 2)
    N = rng.choice((1, 1, rng.randint(2, 8), rng.randint(2, 32)))
    page = min(page, 128)
    tail = _spread(rng, 33, 1000)
    prefix = _spread(rng, page, min(32768, (1 << 28) // (groups * members * Hkv * D)))
    while groups * members * N * Hq * D * prefix > 1.7e10:
        prefix //= 2
    prefix = max(prefix // page, 1) * page
    return dict(op=op, B=groups * members, groups=groups, N=N, Hq=Hq, Hkv=Hkv, D=D, page=page,
                prefix=prefix, longest=prefix + N + tail,
                shortest=prefix + N + rng.randint(0, tail), tree=rng.random() < 0.4,
                dtype=rng.choice(("bf16", "f16")))


def _lengths(case):
    """Cached tokens of each sequence: from the longest down to the shortest."""
    B, hi, lo = case["B"], case["longest"], case["shortest"]
    return [hi - (hi - lo) * b // max(1, B - 1) for b in range(B)]


def _trees(case):
    """Draft trees: parents before children, depth below 16."""
    rng = random.Random(case["N"] * 1000 + case["B"])
    parents, depths = [], []
    for _ in range(case["B"]):
        depth, parent = [1], [-1]
        for n in range(1, case["N"]):
            p = rng.choice([i for i in range(n) if depth[i] < 16])
            parent.append(p)
            depth.append(depth[p] + 1)
        parents.append(parent)
        depths.append(depth)
    return parents, depths


def _path(parent, node):
    path = []
    while node >= 0:
        path.append(node)
        node = parent[node]
    return path[::-1]


_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _quantise(x):
    """Codes (0..15), e4m3 scales (bytes) and the scales' values of x [..., D], 16 channels each."""
    y = torch.nan_to_num(x, nan=0.0).clamp(-2688.0, 2688.0)
    y = y.view(*y.shape[:-1], -1, 16)
    sixth = torch.tensor(1.0 / 6.0, dtype=torch.float32, device=x.device)
    s8 = (y.abs().amax(-1) * sixth).to(torch.float8_e4m3fn)
    s = s8.float()
    r = torch.where(s > 0, 1.0 / s, 0.0)
    t = y * r[..., None]
    a = t.abs()
    mag = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
           + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code = mag + torch.signbit(y).byte() * 8
    return code.reshape(x.shape), s8.view(torch.uint8), s


def _pack(kc, ks, vc, vs):
    """Records [..., R, 36*D] of tokens [..., 32*R, D] of codes and [..., 32*R, D/16] of scales."""
    lead, D = kc.shape[:-2], kc.shape[-1]
    R = kc.shape[-2] // 32
    k = kc.view(*lead, R, 32, D // 32, 16, 2)
    k = (k[..., 0] | (k[..., 1] << 4)).transpose(-3, -2).reshape(*lead, R, 16 * D)
    v = vc.view(*lead, R, 16, 2, D)
    v = (v[..., 0, :] | (v[..., 1, :] << 4)).transpose(-2, -1).reshape(*lead, R, 16 * D)
    sk = ks.reshape(*lead, R, 2 * D)
    sv = vs.view(*lead, R, 32, D // 16).transpose(-2, -1).reshape(*lead, R, 2 * D)
    return torch.cat((k, v, sk, sv), -1)


def _unpack(rec, D):
    """The inverse of _pack, as codes and scale bytes."""
    lead, R = rec.shape[:-2], rec.shape[-2]
    k = rec[..., :16 * D].reshape(*lead, R, D // 32, 32, 16).transpose(-3, -2)
    k = torch.stack((k & 15, k >> 4), -1).reshape(*lead, R * 32, D)
    v = rec[..., 16 * D:32 * D].reshape(*lead, R, D, 16).transpose(-2, -1)
    v = torch.stack((v & 15, v >> 4), -2).reshape(*lead, R * 32, D)
    sk = rec[..., 32 * D:34 * D].reshape(*lead, R * 32, D // 16)
    sv = rec[..., 34 * D:].reshape(*lead, R, D // 16, 32).transpose(-2, -1)
    return k, sk, v, sv.reshape(*lead, R * 32, D // 16)


def _values(code, scale):
    """fp32 values of codes [..., D] with e4m3 scale bytes [..., D/16]."""
    lut = torch.tensor(E2M1 + tuple(-e for e in E2M1), device=code.device)
    s = scale.contiguous().view(torch.float8_e4m3fn).float()
    return (lut[code.int()].view(*scale.shape, 16) * s[..., None]).view(code.shape)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _tokens(rows, T, case, seed):
    """Quantised keys and values of T tokens of `rows` sequences: codes [rows,Hkv,T,D], scales."""
    g = _generator(seed)
    shape = (rows, case["Hkv"], T, case["D"])
    gain = torch.exp(0.5 * torch.randn(shape[1], 1, shape[3], generator=g, device="cuda"))
    kc, ks, _ = _quantise(torch.randn(shape, generator=g, device="cuda") * gain)
    vc, vs, _ = _quantise(torch.randn(shape, generator=g, device="cuda") * 0.7)
    return kc, ks, vc, vs


def _table(case):
    """A page table with the pages of every sequence in random places of the pool: the first
    `shared` pages of each group's are the same ones."""
    page, lens = case["page"], _lengths(case)
    shared = case.get("prefix", 0) // page
    width = max(1, max(-(-n // page) for n in lens))
    held = [-(-n // page) for n in lens]
    groups = case.get("groups", 1)
    n_pages = max(1, sum(h - shared for h in held) + groups * shared + 3)
    order = list(range(n_pages))
    random.Random(n_pages).shuffle(order)
    common = [[order.pop() for _ in range(shared)] for _ in range(groups)]
    per = case["B"] // groups
    table = [common[b // per] + [order.pop() if j < h else -1 for j in range(shared, width)]
             for b, h in enumerate(held)]
    return table, n_pages


def _head_scales(case, g):
    two = 0.5 + torch.rand(2, case["Hkv"], generator=g, device="cuda")
    return two[0].contiguous(), two[1].contiguous()


def _axes(case):
    """Axis of every pair: time, height and width in turn, the last pairs all of time."""
    if case["axes"] == 1:
        return [0] * case["pairs"]
    return [i % 3 if i < 3 * (case["pairs"] * 10 // 32) else 0 for i in range(case["pairs"])]


def _positions(case):
    """Positions [axes][B][N]: text counts on all axes alike; a prompt has an image in it, whose
    tokens stand at one time and go along its rows and columns."""
    lens, N = _lengths(case), case["N"]
    out = [[[0] * N for _ in range(case["B"])] for _ in range(case["axes"])]
    for b, n in enumerate(lens):
        base = n - N
        image = range(N // 8, N // 8 + (N // 2 if N > 64 and case["axes"] == 3 else 0))
        wide = max(1, math.isqrt(len(image)))
        at = max(0, base)
        for i in range(N):
            if i in image:
                y, x = divmod(i - image.start, wide)
                here = (at, at + y, at + x)
                if i + 1 == image.stop:
                    at += max(y, wide - 1) + 1
            else:
                here = (at,) * 3
                at += 1 if base + i >= 0 else 0
            for a in range(case["axes"]):
                out[a][b][i] = here[a]
    return out


def _angles(case):
    """Cosines and sines [positions, 2, pairs], worked out in 64 bits."""
    pos = torch.arange(case["longest"] + 1, dtype=torch.float64, device="cuda")
    freq = BASE ** (-torch.arange(case["pairs"], dtype=torch.float64, device="cuda")
                    / case["pairs"])
    angle = pos[:, None] * freq
    return torch.stack((angle.cos(), angle.sin()), 1).float()


def prepare(case, seed):
    B, N, Hq, Hkv, D, page = (case[k] for k in ("B", "N", "Hq", "Hkv", "D", "page"))
    g = _generator(seed + 1)
    table, n_pages = _table(case)
    s = dict(case=case, kv_len=_int(_lengths(case)), status=_int([0]), table=_int(table))
    s["k_scale"], s["v_scale"] = _head_scales(case, g)
    rec = (Hkv, page // 32, 36 * D)
    # the block's queries, keys and values are slices of the fused projection's output
    qkv = torch.randn(B, N, (Hq + 2 * Hkv) * D, generator=g, device="cuda") * 1.5
    qkv = qkv.to(_DTYPES[case["dtype"]])
    s["q"], s["k"], s["v"] = (t.unflatten(-1, (-1, D))
                              for t in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
    if case["op"] == "rotate":
        s["pages"] = torch.zeros(n_pages, *rec, dtype=torch.uint8, device="cuda")
        s["positions"] = _int(_positions(case))
        s["cos_sin"] = _angles(case)
        s["axis"] = torch.tensor(_axes(case), dtype=torch.uint8, device="cuda")
        return s
    width, shared = s["table"].shape[1], case.get("prefix", 0) // page
    s["pages"] = torch.randint(0, 256, (n_pages, *rec), generator=g, device="cuda",
                               dtype=torch.uint8)
    groups = case.get("groups", 1)
    per = B // groups
    for rows, first, last, places in ((groups, 0, shared, s["table"][::per]),
                                      (B, shared, width, s["table"])):
        if first == last:
            continue
        packed = _pack(*_tokens(rows, (last - first) * page, case, seed + (first > 0)))
        packed = packed.view(rows, Hkv, last - first, page // 32, 36 * D).transpose(1, 2)
        places = places[:, first:last]
        s["pages"][places[places >= 0].long()] = packed[places >= 0]
    s["scale"] = D ** -0.5
    s["parent"] = _int(_trees(case)[0]) if case["tree"] else None
    if case["op"] == "shared":
        s["group"] = _int([i * per for i in range(groups + 1)])
    return s


# ------------------------------------------------------------------ plain forms
def _ancestors(parent):
    """[B,N,N] truth values: node m is on node n's path (n itself among it)."""
    N = parent.shape[1]
    step = (parent[..., None] == torch.arange(N, device=parent.device)).float()
    step = step + torch.eye(N, device=parent.device)
    return torch.linalg.matrix_power(step, max(1, N - 1)) > 0.5


def _plain_attend(s):
    c = s["case"]
    B, N, Hq, Hkv, D = (c[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    rec = s["pages"][s["table"].clamp(min=0).long()]            # [B,width,Hkv,R,36D]
    rec = rec.transpose(1, 2).flatten(2, 3)
    kc, ks, vc, vs = _unpack(rec, D)
    T = kc.shape[2]
    pos = torch.arange(T, device="cuda")[None, None, :]
    base = (s["kv_len"] - N)[:, None, None]
    u = pos - base                                              # position within the block
    n = torch.arange(N, device="cuda")[None, :, None]
    if s["parent"] is None:
        seen = u <= n
        index, entry = base + n, pos                            # on the node's path
    else:
        path = _ancestors(s["parent"])
        inside = torch.gather(path, 2, u.clamp(0, N - 1).expand(B, N, T))
        seen = (u < 0) | ((u < N) & inside)
        depth = path.sum(2) - 1
        index = base + depth[:, :, None]
        entry = torch.where(u < 0, pos, base + torch.gather(
            depth[:, None, :], 2, u.clamp(0, N - 1)))
    if c["op"] == "window":
        seen = seen & ((entry > index - c["window"]) | (entry < c["sinks"]))
    seen = (seen & (n >= -base))[:, None, :, None, :]
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).transpose(1, 2)
    q = q.reshape(B, Hkv, N * (Hq // Hkv), D) * (s["scale"] * s["k_scale"])[None, :, None, None]
    x = (q @ _values(kc, ks).transpose(-2, -1)).view(B, Hkv, N, Hq // Hkv, T)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    v = _values(vc, vs).masked_fill((pos >= s["kv_len"][:, None, None])[..., None], 0.0)
    o = p.view(B, Hkv, -1, T) @ v
    o = o.view(B, Hkv, N, Hq // Hkv, D) / total.masked_fill(total == 0, 1.0)
    o = o * s["v_scale"][None, :, None, None, None]
    return o.transpose(1, 2).reshape(B, N, Hq, D).to(s["q"].dtype)


def _slots(s, first, count):
    """Page, record and place of `count` positions from `first` [B] on, and which exist."""
    page = s["case"]["page"]
    pos = first[:, None] + torch.arange(count, device="cuda")[None, :]
    at = pos.clamp(min=0)
    where = torch.gather(s["table"], 1, (at // page).long()).clamp(min=0)
    return where.long(), (at % page // 32).long(), at % 32, pos >= 0


def _rotated(s, x):
    """x [B,N,H,D] in fp32 with its pairs turned by their positions."""
    c = s["case"]
    P = c["pairs"]
    where = s["positions"].long()[s["axis"].long()].permute(1, 2, 0)       # [B,N,pairs]
    i = torch.arange(P, device="cuda")
    cos, sin = (s["cos_sin"][where, j, i][:, :, None] for j in (0, 1))
    x = x.float()
    turn, rest = x[..., :2 * P], x[..., 2 * P:]
    if c["adjacent"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turn[..., :P], turn[..., P:]
        turn = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turn, rest), -1)


def _plain_rotate(s):
    c = s["case"]
    B, N, Hkv, D, page = (c[k] for k in ("B", "N", "Hkv", "D", "page"))
    inverse = [(1.0 / s[n])[None, None, :, None] for n in ("k_scale", "v_scale")]
    kc, ks, _ = _quantise(_rotated(s, s["k"]) * inverse[0])
    vc, vs, _ = _quantise(s["v"].float() * inverse[1])
    # the records around the block: unpacked, the block's tokens put in, packed again
    base = s["kv_len"] - N
    first = base.clamp(min=0) // 32
    last = (s["kv_len"] - 1) // 32
    held = first[:, None] + torch.arange(-(-N // 32) + 1, device="cuda")[None, :]
    b, r = torch.nonzero(held <= last[:, None], as_tuple=True)
    t = held[b, r] * 32
    where = s["table"][b, (t // page).long()].long()
    place = (t % page // 32).long()
    old = _unpack(s["pages"][where, :, place][:, :, None], D)   # [M,Hkv,32,...]
    n = t[:, None] + torch.arange(32, device="cuda")[None, :] - base[b][:, None]
    mine = ((n >= 0) & (n < N))[:, None, :, None]
    at = n.clamp(0, N - 1).long()
    new = [torch.where(mine, a[b[:, None], at].transpose(1, 2), o)
           for a, o in zip((kc, ks, vc, vs), old)]
    s["pages"][where, :, place] = _pack(*new)[:, :, 0]
    # and read back
    where, place, slot, there = _slots(s, base, N)
    rec = s["pages"][where, :, place]                           # [B,N,Hkv,36D]
    i = slot[..., None, None].long().expand(B, N, Hkv, 1)
    kb = rec[..., :16 * D].view(B, N, Hkv, D // 32, 32, 16)
    kb = torch.gather(kb, 4, i[..., None, None].expand(B, N, Hkv, D // 32, 1, 16))[..., 0, :]
    kcode = torch.stack((kb & 15, kb >> 4), -1).view(B, N, Hkv, D)
    vb = rec[..., 16 * D:32 * D].view(B, N, Hkv, D, 16)
    vb = torch.gather(vb, 4, (i // 2)[..., None].expand(B, N, Hkv, D, 1))[..., 0]
    vcode = torch.where(i % 2 == 0, vb & 15, vb >> 4)
    sk = rec[..., 32 * D:34 * D].view(B, N, Hkv, 32, D // 16)
    sk = torch.gather(sk, 3, i[..., None].expand(B, N, Hkv, 1, D // 16))[..., 0, :]
    sv = rec[..., 34 * D:].view(B, N, Hkv, D // 16, 32)
    sv = torch.gather(sv, 4, i[..., None].expand(B, N, Hkv, D // 16, 1))[..., 0]
    there = there[..., None, None]
    k = _values(kcode, sk) * s["k_scale"][:, None]
    v = _values(vcode, sv) * s["v_scale"][:, None]
    q = torch.where(there, _rotated(s, s["q"]), 0.0).to(s["q"].dtype)
    return q, torch.where(there, k, 0.0), torch.where(there, v, 0.0)


# ------------------------------------------------------------------ the framework's calls
def _bind(s):
    """The calls of one pass, bound to the program's buffers as a serving loop does."""
    import hybrid_gated_deltanet_delta_gb300 as gdn

    c = s["case"]
    sizes = [c[k] for k in ("B", "N", "Hq", "Hkv", "D")]
    kw = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], status=s["status"])
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    where = (s["pages"], s["table"], s["kv_len"])
    if c["op"] == "rotate":
        ko, vo = (torch.empty(s["k"].shape, device="cuda") for _ in range(2))
        return [gdn.bind_kv4_append_rotary(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"],
                                           *where, out, axis=s["axis"], adjacent=c["adjacent"],
                                           **kw),
                gdn.bind_kv4_read(*where, ko, vo, **kw)], (out, ko, vo)
    kw.update(scale=s["scale"], parent=s["parent"])
    if c["op"] == "window":
        ws = torch.empty(gdn.gdn_kv4_attention_workspace_bytes(*sizes), dtype=torch.uint8,
                         device="cuda")
        return [gdn.bind_kv4_attention_window(s["q"], *where, out, ws, window=c["window"],
                                              sinks=c["sinks"], **kw)], out
    ws = torch.empty(gdn.gdn_kv4_attention_shared_workspace_bytes(*sizes, c["groups"]),
                     dtype=torch.uint8, device="cuda")
    return [gdn.bind_kv4_attention_shared(s["q"], *where, s["group"], out, ws, **kw)], out


def run(s):
    if own:
        if "calls" not in s:
            s["calls"], s["out"] = _bind(s)
        for call in s["calls"]:
            call()
        return s["out"]
    return _plain_rotate(s) if s["case"]["op"] == "rotate" else _plain_attend(s)


# ------------------------------------------------------------------ what it cannot do without
def work(case):
    B, N, Hq, Hkv, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    lens = _lengths(case)
    token = Hkv * 9 * D // 8                                   # K and V codes and scales
    if case["op"] == "rotate":
        rows = sum(min(N, n) for n in lens)
        size = 4 if case["dtype"] == "f32" else 2
        # the projections and angles in, queries out, records out and in, stored values out
        return {"bytes": rows * ((Hq + 2 * Hkv) * D * size + 2 * token + 4 * case["axes"]
                                 + 8 * case["pairs"]) + B * N * Hq * D * size
                + B * N * 2 * Hkv * D * 4,
                "flops": 4.0 * rows * 2 * Hkv * D + 6.0 * rows * (Hq + Hkv) * case["pairs"]}
    depths = _trees(case)[1] if case["tree"] else None
    window, sinks = case.get("window", 1 << 40), case.get("sinks", 0)
    tokens = pairs = 0
    for b, length in enumerate(lens):
        base = length - N
        most = N if depths is None else max(depths[b])
        tokens += min(length, min(sinks, base) + window + most - 1 + N - most
                      if base >= 0 else length)
        for n in range(max(0, -base), N):
            seen = base + (n + 1 if depths is None else depths[b][n])
            pairs += max(0, min(seen, window + min(sinks, max(0, seen - window))))
    if case["op"] == "shared":
        per = B // case["groups"]
        tokens -= case["prefix"] * case["groups"] * (per - 1)
    return {"bytes": tokens * token + 2 * 2 * B * N * Hq * D + 4 * len(lens),
            "flops": 4.0 * D * Hq * pairs}


# ------------------------------------------------------------------ 64-bit values
_E4M3 = np.array([(-1.0) ** (b >> 7) * (2.0 ** -6 * (b & 7) / 8 if not b >> 3 & 15 else
                                        2.0 ** ((b >> 3 & 15) - 7) * (1 + (b & 7) / 8))
                  if b & 127 != 127 else math.nan for b in range(256)])


def _double(rec, D):
    """float64 keys and values [R*32,D] of one head's records [R,36D], each looked up by the place
    of its code and of its scale."""
    R = rec.shape[0]
    grid = torch.tensor(E2M1 + tuple(-e for e in E2M1), dtype=torch.float64, device="cuda")
    scales = torch.from_numpy(_E4M3).cuda()
    t = torch.arange(32, device="cuda")[:, None]
    ch = torch.arange(D, device="cuda")[None, :]
    out = []
    for at, high, scale in ((ch // 32 * 512 + t * 16 + ch % 32 // 2, ch % 2,
                             32 * D + t * (D // 16) + ch // 16),
                            (16 * D + ch * 16 + t // 2, t % 2, 34 * D + ch // 16 * 32 + t)):
        code = rec[:, at].int() >> (4 * high) & 15
        out.append((grid[code] * scales[rec[:, scale].int()]).view(R * 32, D))
    return out


def _exact_rotate(case, s):
    B, N, P = case["B"], case["N"], case["pairs"]
    lens, axis = _lengths(case), _axes(case)
    first = torch.tensor([2 * i if case["adjacent"] else i for i in range(P)], device="cuda")
    second = first + (1 if case["adjacent"] else P)
    rows = [s["positions"][a].long() for a in axis]             # of each pair, [B,N]
    cs = torch.stack([s["cos_sin"][rows[i]][..., i].double() for i in range(P)], -1)

    def turned(x):
        x = x.double()
        out = x.clone()
        a, b, c, d = x[..., first], x[..., second], cs[:, :, None, 0], cs[:, :, None, 1]
        out[..., first] = a * c - b * d
        out[..., second] = a * d + b * c
        return out

    q = turned(s["q"])
    out = []
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    steps = torch.from_numpy(_E4M3[:127]).to("cuda")
    for x, gs in ((turned(s["k"]), s["k_scale"]), (s["v"].double(), s["v_scale"])):
        gs = gs.double()[None, None, :, None]
        y = (x / gs).clamp(-2688, 2688).unflatten(-1, (-1, 16))
        want = y.abs().amax(-1) / 6
        hi = torch.searchsorted(steps, want).clamp(1, 126)
        lo = hi - 1
        up = (want - steps[lo] > steps[hi] - want) | \
            ((want - steps[lo] == steps[hi] - want) & (hi % 2 == 0))
        scale = torch.where(up, steps[hi], steps[lo])[..., None]
        a = torch.where(scale > 0, y.abs() / scale, 0.0).clamp(max=6.0)
        hi = torch.searchsorted(grid, a).clamp(1, 7)
        lo = hi - 1
        up = (a - grid[lo] > grid[hi] - a) | ((a - grid[lo] == grid[hi] - a) & (hi % 2 == 0))
        mag = torch.where(up, grid[hi], grid[lo]) * scale
        out.append(torch.where(y < 0, -mag, mag).flatten(-2) * gs)
    for b, n in enumerate(lens):
        for t in (q, *out):
            t[b, :max(0, N - n)] = 0
    return (q, *out)


def exact(case, seed):
    B, N, Hq, Hkv, D, page = (case[k] for k in ("B", "N", "Hq", "Hkv", "D", "page"))
    if case["op"] == "rotate":
        return _exact_rotate(case, prepare(case, seed))
    if 4.0 * B * N * Hq * D * case["longest"] > 5e11 or B * Hkv * D * case["longest"] > 1.5e9:
        return None
    s = prepare(case, seed)
    G, lens = Hq // Hkv, _lengths(case)
    window, sinks = case.get("window", 1 << 40), case.get("sinks", 0)
    parents = _trees(case)[0] if case["tree"] else None
    o = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        base = length - N
        if length == 0:
            continue
        seen = torch.zeros(N, length, dtype=torch.bool)
        for n in range(max(0, -base), N):
            # the entries of the node's path, and which of them are first or last enough
            block = range(n + 1) if parents is None else _path(parents[b], n)
            end = base + len(block)
            seen[n, :min(max(0, base), sinks)] = True
            seen[n, max(0, end - window):max(0, base)] = True
            for i, m in enumerate(block):
                if base + m >= 0 and (base + i >= end - window or base + i < sinks):
                    seen[n, base + m] = True
        seen = seen.cuda()
        row = s["pages"][s["table"][b, :-(-length // page)].long()]        # [pages,Hkv,R,36D]
        for h in range(Hkv):
            k, v = _double(row[:, h].reshape(-1, 36 * D), D)
            k, v = (k[:length] * s["k_scale"][h].double(), v[:length] * s["v_scale"][h].double())
            for i in range(G):
                x = s["q"][b, :, h * G + i].double() @ k.T * s["scale"]
                x = torch.where(seen, x, -math.inf)
                top = x.amax(1, keepdim=True)
                p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
                total = p.sum(1, keepdim=True)
                o[b, :, h * G + i] = (p @ v) / torch.where(total > 0, total, 1.0)
    return o
