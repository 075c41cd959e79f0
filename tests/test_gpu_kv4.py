"""4-bit key/value cache on the GPU against the 64-bit reference: append and
read back, attention, commit of accepted paths, and the page pool."""
import numpy as np
import pytest

import kv4_reference as ref
from gpu_helpers import torch

pytestmark = pytest.mark.gpu

# torch type and unit roundoff (half a unit in the last of 8 and 11 significand bits)
DT = {"bf16": ("bfloat16", 2.0 ** -8), "f16": ("float16", 2.0 ** -11), "f32": ("float32", 0.0)}


def tdtype(name):
    return getattr(torch(), DT[name][0])


def cuda(a):
    return torch().from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return cuda(np.asarray(a, np.int32))


def status_word():
    return torch().zeros(1, dtype=torch().int32, device="cuda")


class Setup:
    """A cache of random garbage pages, a table over random pages, and scales."""

    def __init__(self, rng, lens, H, D, P, slack=0, layers=None, ones=False):
        self.H, self.D, self.P, self.lens = H, D, P, np.asarray(lens)
        held = [-(-(n + slack) // P) for n in lens]
        self.width = max(1, max(held)) + 1
        n_pages = sum(held) + 2
        order = rng.permutation(n_pages)
        self.table = np.full((len(lens), self.width), -1, np.int64)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = order[at:at + h]
            at += h
        shape = (n_pages, H, P // 32, 36 * D)
        self.pages = rng.integers(0, 256, ((layers,) if layers else ()) + shape, dtype=np.uint8)
        self.ks = np.ones(H, np.float32) if ones else rng.uniform(0.3, 2, H).astype(np.float32)
        self.vs = np.ones(H, np.float32) if ones else rng.uniform(0.3, 2, H).astype(np.float32)

    def gpu(self):
        self.g_pages, self.g_table = cuda(self.pages), i32(self.table)
        self.g_len, self.g_ks, self.g_vs = i32(self.lens), cuda(self.ks), cuda(self.vs)
        self.status = status_word()
        return dict(k_scale=self.g_ks, v_scale=self.g_vs, status=self.status)

    def fill(self, rng, scale=1.0):
        """Quantised random tokens at every position of every sequence (reference side)."""
        cache = ref.Cache(self.pages, self.D)
        for b, n in enumerate(self.lens):
            shape = (int(n), self.H, self.D)
            kc, ks = ref.quantise(scale * rng.standard_normal(shape), self.ks)
            vc, vs = ref.quantise(rng.standard_normal(shape), self.vs)
            for p in range(int(n)):
                for h in range(self.H):
                    cache.put(self.table[b, p // self.P], h, p % self.P, kc[p, h], ks[p, h],
                              vc[p, h], vs[p, h])
        return cache


def rand_trees(rng, B, N, depth=16):
    out = np.zeros((B, N), np.int64)
    for b in range(B):
        d = [1]
        out[b, 0] = -1
        for n in range(1, N):
            out[b, n] = rng.choice([i for i in range(n) if d[i] < depth])
            d.append(d[out[b, n]] + 1)
    return out


# ------------------------------------------------------------------ append, read
@pytest.mark.parametrize("dtype, lens, N, H, D, P", [
    ("bf16", [1], 1, 1, 64, 32),
    ("bf16", [33, 64, 31], 1, 2, 256, 32),
    ("f16", [40, 16, 97], 16, 4, 128, 64),
    ("f32", [0, 5, 22, 23, 200], 22, 2, 64, 96),      # absent, shorter than the block
    ("bf16", [300], 300, 1, 256, 64),                 # a whole prompt, odd end
    ("f32", [161, 130], 65, 3, 128, 32),
    ("f16", [64], 32, 2, 256, 1664),
])
def test_append_and_read(gpu_lib, dtype, lens, N, H, D, P):
    rng, t = np.random.default_rng(N * D + H), torch()
    s = Setup(rng, lens, H, D, P)
    kw = s.gpu()
    # k and v as slices of one fused projection: strided by batch and node
    qkv = t.from_numpy(rng.standard_normal((len(lens), N, 3 * H * D))).cuda().to(tdtype(dtype))
    k = qkv[..., H * D:2 * H * D].unflatten(-1, (H, D))
    v = qkv[..., 2 * H * D:].unflatten(-1, (H, D))
    gpu_lib.gdn_kv4_append(k, v, s.g_pages, s.g_table, s.g_len, **kw)
    ko, vo = (t.full((len(lens), N, H, D), 7.0, device="cuda") for _ in range(2))
    gpu_lib.gdn_kv4_read(s.g_pages, s.g_table, s.g_len, ko, vo, **kw)
    out16 = [t.empty(ko.shape, dtype=t.bfloat16, device="cuda") for _ in range(2)]
    gpu_lib.gdn_kv4_read(s.g_pages, s.g_table, s.g_len, *out16, **kw)
    assert int(s.status.item()) == 0
    cache = ref.Cache(s.pages, D)
    ref.append(cache, s.table, s.lens, P, k.float().cpu().numpy(), v.float().cpu().numpy(), s.ks,
               s.vs)
    # bit for bit: the block's bytes, and every byte that is not the block's
    assert np.array_equal(s.g_pages.cpu().numpy(), s.pages)
    for b, n in enumerate(s.lens):
        for i in range(N):
            p = int(n) - N + i
            for h in range(H):
                if p < 0:
                    assert not ko[b, i, h].any() and not vo[b, i, h].any()
                    continue
                kc, ks, vc, vs = cache.get(s.table[b, p // P], h, p % P)
                # code * scale is exact; the head scale's product is rounded once
                want = (ref.values(kc, ks).astype(np.float32) * s.ks[h],
                        ref.values(vc, vs).astype(np.float32) * s.vs[h])
                assert np.array_equal(ko[b, i, h].cpu().numpy(), want[0])
                assert np.array_equal(vo[b, i, h].cpu().numpy(), want[1])
    for full, half in zip((ko, vo), out16):
        assert t.equal(full.to(t.bfloat16), half)


def test_append_special_values(gpu_lib):
    """Zeros, ties, subnormal scales, saturation; NaN and infinity are stored finite, reported."""
    rng, t = np.random.default_rng(3), torch()
    D = 64
    s = Setup(rng, [6], 1, D, 32, ones=True)
    kw = s.gpu()
    x = np.zeros((1, 6, 1, D), np.float32)
    x[0, 1, 0, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -0.75, -1.25, -1.75, -2.5,
                       -3.5, -5, -6]
    x[0, 1, 0, 16:32] = 1e-6                       # scale rounds to 0
    x[0, 1, 0, 32:48] = np.linspace(-0.012, 0.012, 16)   # subnormal scale
    x[0, 1, 0, 48:] = np.linspace(-1e5, 1e5, 16)   # beyond +-2688
    x[0, 2, 0, :16] = -0.0
    x[0, 3, 0] = rng.standard_normal(D) * 10.0 ** rng.uniform(-4, 3, D)
    finite = x.copy()
    for trial, bad in enumerate((None, np.nan, np.inf, -np.inf)):
        a = finite.copy()
        if bad is not None:
            a[0, 4, 0, 5] = bad
        s.status.zero_()
        gpu_lib.gdn_kv4_append(cuda(a), cuda(a), s.g_pages, s.g_table, s.g_len, **kw)
        cache = ref.Cache(s.pages, D)
        ref.append(cache, s.table, s.lens, 32, a, a, s.ks, s.vs)
        assert np.array_equal(s.g_pages.cpu().numpy(), s.pages)
        assert int(s.status.item()) == (0 if bad is None else gpu_lib.GDN_ERR_NONFINITE)


def test_append_on_its_own_stream_and_in_a_graph(gpu_lib):
    """A captured append follows the lengths that the buffer holds at replay."""
    rng, t = np.random.default_rng(4), torch()
    s = Setup(rng, [40, 70], 2, 128, 32, slack=40)
    kw = s.gpu()
    k = t.from_numpy(rng.standard_normal((2, 3, 2, 128))).cuda().to(t.bfloat16)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        call = gpu_lib.bind_kv4_append(k, k, s.g_pages, s.g_table, s.g_len, **kw)
        call()
        side.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            gpu_lib.gdn_kv4_append(k, k, s.g_pages, s.g_table, s.g_len, **kw)
    cache = ref.Cache(s.pages, 128)
    kn = k.float().cpu().numpy()
    ref.append(cache, s.table, s.lens, 32, kn, kn, s.ks, s.vs)
    for step in (1, 2):
        s.g_len += 3
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        ref.append(cache, s.table, s.lens + 3 * step, 32, kn, kn, s.ks, s.vs)
    assert np.array_equal(s.g_pages.cpu().numpy(), s.pages)


def test_lengths_and_pages_out_of_range_are_reported(gpu_lib):
    rng, t = np.random.default_rng(5), torch()
    s = Setup(rng, [40, 40], 1, 64, 32)
    kw = s.gpu()
    before = s.g_pages.clone()
    k = t.ones(2, 2, 1, 64, device="cuda")
    ko, vo = t.full_like(k, 9), t.full_like(k, 9)
    q = t.ones(2, 2, 2, 64, device="cuda", dtype=t.bfloat16)
    o = t.full_like(q, 9)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(2, 2, 2, 1, 64), dtype=t.uint8,
                 device="cuda")
    for bad in (-1, s.width * 32 + 1):
        n = i32([bad, bad])
        for fn, args in ((gpu_lib.gdn_kv4_append, (k, k, s.g_pages, s.g_table, n)),
                         (gpu_lib.gdn_kv4_read, (s.g_pages, s.g_table, n, ko, vo))):
            s.status.zero_()
            fn(*args, **kw)
            assert int(s.status.item()) == gpu_lib.GDN_ERR_ROW_RANGE
        s.status.zero_()
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, n, o, ws, scale=0.1, **kw)
        assert int(s.status.item()) == gpu_lib.GDN_ERR_ROW_RANGE
        assert not o.any() and not ko.any() and not vo.any()
    for page in (-1, s.pages.shape[0]):
        s.g_table[0, 1] = page
        for fn, args, more in (
                (gpu_lib.gdn_kv4_append, (k[:1], k[:1], s.g_pages, s.g_table[:1], s.g_len[:1]), {}),
                (gpu_lib.gdn_kv4_read, (s.g_pages, s.g_table[:1], s.g_len[:1], ko[:1], vo[:1]), {}),
                (gpu_lib.gdn_kv4_attention, (q[:1], s.g_pages, s.g_table[:1], s.g_len[:1], o[:1],
                                             ws), dict(scale=0.1))):
            s.status.zero_()
            fn(*args, **more, **kw)
            assert int(s.status.item()) == gpu_lib.GDN_ERR_PAGE_RANGE
        assert not ko[0].any()
    assert t.equal(s.g_pages, before)


# ------------------------------------------------------------------ attention
def check_attention(gpu_lib, s, cache, q, dtype, scale, parent=None, stream=None):
    t = torch()
    B, N, Hq, D = q.shape
    kw = s.gpu()
    o = t.full((B, N, Hq, D), 5.0, dtype=tdtype(dtype), device="cuda")
    lse = t.full((B, N, Hq), 5.0, device="cuda")
    ws = t.full((gpu_lib.gdn_kv4_attention_workspace_bytes(B, N, Hq, s.H, D),), 255,
                dtype=t.uint8, device="cuda")
    par = None if parent is None else i32(parent)
    for _ in range(2):   # the workspace as a call leaves it serves the next one
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=scale,
                                  parent=par, lse=lse, **kw)
    assert int(s.status.item()) == 0
    want, wlse, weight, reach = ref.attention(cache, s.table, s.lens, s.P,
                                              q.double().cpu().numpy(), scale, s.ks, s.vs, parent)
    # Error bound.  The logits are fp32 sums of D exact products (D * 2^-23 of the
    # sum of magnitudes, `reach`), scaled and exponentiated in fp32 (a few 2^-22 of
    # a logit of size <= reach), which moves every probability by at most `d`
    # relatively and the result by 2 d of the weighted magnitudes; probabilities are
    # rounded to binary16 (2^-11 relative, 2^-25 absolute each, against a sum of at
    # least 2^-8 of the largest); fp32 sums over T positions add T * 2^-23; the
    # output is rounded once.
    T = max(1, int(s.lens.max()))
    d = (D * 2.0 ** -23 + 2.0 ** -20) * reach + 2.0 ** -20
    vmax = np.abs(want).max() + weight.max()
    tol = (DT[dtype][1] * np.abs(want)
           + weight * (2 * d[..., None] + 2.0 ** -11 + T * 2.0 ** -22)
           + T * 2.0 ** -25 * vmax + 2.0 ** -24)
    err = np.abs(o.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"worst {(err / tol).max():.3f} of the bound"
    l = lse.double().cpu().numpy()
    assert np.array_equal(np.isinf(l), np.isinf(wlse))
    seen = np.isfinite(wlse)
    ltol = (d + T * 2.0 ** -22)[seen] + 2.0 ** -22 * np.abs(wlse[seen])
    assert (np.abs(l[seen] - wlse[seen]) <= ltol).all()
    return o, lse


ATTEND = [
    # dtype, lens, N, Hq, H, D, P, tree
    ("bf16", [1], 1, 1, 1, 64, 32, False),
    ("bf16", [700], 1, 24, 4, 256, 64, False),
    ("f16", [0, 1, 31, 32, 33, 129, 300], 1, 8, 2, 128, 32, False),
    ("bf16", [127, 128, 129, 255, 257], 1, 6, 1, 64, 96, False),
    ("bf16", [16, 17, 150, 400], 16, 12, 2, 256, 128, False),
    ("f16", [5, 0, 22, 260], 16, 8, 8, 128, 64, False),   # blocks with absent nodes
    ("bf16", [22, 150, 513], 22, 24, 4, 256, 64, True),
    ("f16", [64, 65, 300], 64, 4, 4, 64, 32, True),
    ("bf16", [3, 40, 0], 7, 16, 2, 128, 96, True),          # trees with absent nodes
    ("bf16", [200], 200, 6, 2, 256, 64, False),             # a prompt from nothing
    ("f16", [391], 133, 10, 2, 128, 1664, False),
    ("bf16", [150, 90], 90, 3, 1, 64, 32, False),
    ("bf16", [333], 5, 40, 2, 256, 64, False),              # 100 rows of a kv head
    ("f16", [1000, 40], 2, 34, 2, 128, 64, False),
]


@pytest.mark.parametrize("dtype, lens, N, Hq, H, D, P, tree", ATTEND)
def test_attention(gpu_lib, dtype, lens, N, Hq, H, D, P, tree):
    rng, t = np.random.default_rng(sum(lens) + N * D + Hq), torch()
    s = Setup(rng, lens, H, D, P)
    cache = s.fill(rng)
    parent = rand_trees(rng, len(lens), N) if tree else None
    qkv = t.from_numpy(rng.standard_normal((len(lens), N, (Hq + 2) * D))).cuda().to(tdtype(dtype))
    q = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
    check_attention(gpu_lib, s, cache, q, dtype, D ** -0.5, parent)


@pytest.mark.parametrize("gain", [0.0, 30.0, 1000.0])
def test_attention_logit_range(gpu_lib, gain):
    """Equal logits, and logits whose running maximum rises by hundreds along the cache."""
    rng, t = np.random.default_rng(8), torch()
    s = Setup(rng, [600, 350], 2, 128, 64)
    cache = s.fill(rng)
    q = (t.from_numpy(rng.standard_normal((2, 4, 6, 128))) * gain).cuda().to(t.bfloat16)
    check_attention(gpu_lib, s, cache, q, "bf16", 128 ** -0.5)


@pytest.mark.parametrize("size", [1e-30, 1e-5, 1e4, 1e30])
def test_attention_query_magnitudes(gpu_lib, size):
    """bf16 queries far outside binary16's range; the scale brings the logits back."""
    rng, t = np.random.default_rng(9), torch()
    s = Setup(rng, [200], 1, 64, 32)
    cache = s.fill(rng)
    q = (t.from_numpy(rng.standard_normal((1, 3, 4, 64))) * size).cuda().to(t.bfloat16)
    check_attention(gpu_lib, s, cache, q, "bf16", 0.125 / size)


def test_attention_infinite_and_nan_queries_stay_in_their_row(gpu_lib):
    rng, t = np.random.default_rng(10), torch()
    s = Setup(rng, [150], 1, 64, 32)
    s.fill(rng)
    kw = s.gpu()
    q = t.from_numpy(rng.standard_normal((1, 4, 8, 64))).cuda().to(t.bfloat16)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(1, 4, 8, 1, 64), dtype=t.uint8,
                 device="cuda")
    outs = []
    for bad in (None, float("nan"), float("inf")):
        x = q.clone()
        if bad is not None:
            x[0, 1, 3, 7] = bad
        o = t.empty_like(x)
        gpu_lib.gdn_kv4_attention(x, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.1, **kw)
        outs.append(o)
    for o in outs[1:]:
        assert t.isnan(o[0, 1, 3]).any()
        o[0, 1, 3] = outs[0][0, 1, 3]
        assert t.equal(o, outs[0])


def test_attention_bad_tree_is_skipped_and_reported(gpu_lib):
    rng, t = np.random.default_rng(11), torch()
    s = Setup(rng, [100, 100], 1, 64, 32)
    s.fill(rng)
    kw = s.gpu()
    q = t.ones(2, 3, 2, 64, device="cuda", dtype=t.bfloat16)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(2, 3, 2, 1, 64), dtype=t.uint8,
                 device="cuda")
    for bad in ([0, 0, 1], [-1, 1, 0], [-1, 0, -1], [-1, 0, 2]):
        o = t.full_like(q, 4)
        s.status.zero_()
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.1,
                                  parent=i32([bad, [-1, 0, 1]]), **kw)
        assert int(s.status.item()) == gpu_lib.GDN_ERR_BAD_TREE
        assert not o[0].any() and o[1].any()


def test_attention_past_32_bit_offsets(gpu_lib):
    """Pages beyond 4 GiB of the pool."""
    rng, t = np.random.default_rng(12), torch()
    s = Setup(rng, [130], 4, 256, 64)
    cache = s.fill(rng)
    small = s.pages
    n_pages = (5 << 30) // small[0].size
    q = t.from_numpy(rng.standard_normal((1, 2, 8, 256))).cuda().to(t.bfloat16)
    big = t.empty((n_pages, *small.shape[1:]), dtype=t.uint8, device="cuda")
    where = n_pages - 1 - s.table[0]
    for j in range(-(-130 // 64)):
        big[int(where[j])] = cuda(small[s.table[0, j]])
    kw = s.gpu()
    o, o2 = t.empty_like(q), t.empty_like(q)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(1, 2, 8, 4, 256), dtype=t.uint8,
                 device="cuda")
    gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.06, **kw)
    gpu_lib.gdn_kv4_attention(q, big, i32(where[None]), s.g_len, o2, ws, scale=0.06, **kw)
    k = t.empty(1, 130, 4, 256, device="cuda")
    v, k2, v2 = t.empty_like(k), t.empty_like(k), t.empty_like(k)
    gpu_lib.gdn_kv4_read(s.g_pages, s.g_table, s.g_len, k, v, **kw)
    gpu_lib.gdn_kv4_read(big, i32(where[None]), s.g_len, k2, v2, **kw)
    assert int(s.status.item()) == 0
    assert t.equal(o, o2) and t.equal(k, k2) and t.equal(v, v2) and o.any()


def test_attention_repeats_bit_for_bit(gpu_lib):
    rng, t = np.random.default_rng(13), torch()
    s = Setup(rng, [5000, 77, 2300], 2, 128, 64)
    kw = s.gpu()
    k = t.randn(3, 5000, 2, 128, device="cuda")
    gpu_lib.gdn_kv4_append(k, k, s.g_pages, s.g_table, s.g_len, **kw)
    q = t.randn(3, 3, 8, 128, device="cuda").to(t.bfloat16)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(3, 3, 8, 2, 128), dtype=t.uint8,
                 device="cuda")
    outs = []
    for _ in range(5):
        o = t.empty_like(q)
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.09, **kw)
        outs.append(o)
    assert int(s.status.item()) == 0
    assert all(t.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("lens, N, Hq, H, D, P", [
    ([40000], 1, 6, 1, 256, 64),
    ([9000] * 3 + [20011], 16, 12, 2, 256, 64),
    ([3000 + 7 * i for i in range(40)], 1, 16, 4, 64, 32),
    ([2500], 900, 6, 1, 128, 128),
    ([130 + i for i in range(300)], 1, 8, 2, 128, 32),
])
def test_attention_long_and_many(gpu_lib, lens, N, Hq, H, D, P):
    """Sizes that spread a row over many blocks, or many rows over one, against a
    float64 evaluation on the GPU from the stored values (gdn_kv4_read)."""
    rng, t = np.random.default_rng(len(lens) + N), torch()
    s = Setup(rng, lens, H, D, P)
    kw = s.gpu()
    T = max(lens)
    x = t.randn(2, len(lens), T, H, D, device="cuda", dtype=t.bfloat16)
    gpu_lib.gdn_kv4_append(x[0], x[1], s.g_pages, s.g_table, s.g_len, **kw)
    k, v = (t.empty(len(lens), T, H, D, device="cuda") for _ in range(2))
    gpu_lib.gdn_kv4_read(s.g_pages, s.g_table, s.g_len, k, v, **kw)
    q = t.randn(len(lens), N, Hq, D, device="cuda").to(t.bfloat16)
    o = t.empty_like(q)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(len(lens), N, Hq, H, D),
                 dtype=t.uint8, device="cuda")
    scale = D ** -0.5
    gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=scale, **kw)
    assert int(s.status.item()) == 0
    G = Hq // H
    for b, n in enumerate(lens):
        kb, vb = k[b, T - n:].double(), v[b, T - n:].double()      # right-aligned
        hide = t.arange(n, device="cuda")[None] > n - N + t.arange(N, device="cuda")[:, None]
        for h in range(Hq):
            p = (q[b, :, h].double() @ kb[:, h // G].T * scale).masked_fill(hide, -float("inf"))
            p = t.softmax(p, -1)
            want, weight = p @ vb[:, h // G], p @ vb[:, h // G].abs()
            reach = scale * float((q[b, :, h].double().abs() @ kb[:, h // G].abs().T).max())
            d = (D * 2.0 ** -23 + 2.0 ** -20) * reach + 2.0 ** -20
            tol = 2.0 ** -8 * want.abs() + weight * (2 * d + 2.0 ** -11 + n * 2.0 ** -22) \
                + n * 2.0 ** -25 * 12 + 2.0 ** -24
            err = (o[b, :, h].double() - want).abs()
            assert bool((err <= tol).all()), f"sequence {b}: {float((err / tol).max()):.3f}"


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("lens, N, H, D, P, layers, tree", [
    ([22, 70, 200], 22, 2, 256, 64, 3, True),
    ([64, 95, 127, 96], 64, 3, 128, 32, 2, True),
    ([40, 41], 5, 1, 64, 96, 1, True),
    ([1, 33], 1, 1, 64, 32, 2, True),
    ([16, 50], 16, 2, 128, 64, 2, False),
])
def test_commit(gpu_lib, lens, N, H, D, P, layers, tree):
    rng = np.random.default_rng(N + D)
    for trial in range(4):
        s = Setup(rng, lens, H, D, P, layers=layers)
        s.gpu()
        parent = rand_trees(rng, len(lens), N) if tree else None
        accept = rng.integers(0, N, len(lens))
        out = i32(np.full(len(lens), -7))
        gpu_lib.gdn_kv4_commit(s.g_pages, s.g_table, s.g_len, i32(accept), out, N=N,
                               parent=None if parent is None else i32(parent), status=s.status)
        want = ref.commit([ref.Cache(s.pages[l], D) for l in range(layers)], s.table, s.lens, P,
                          N, accept, parent)
        assert int(s.status.item()) == 0
        assert np.array_equal(out.cpu().numpy(), want)
        got = s.g_pages.cpu().numpy()
        for l in range(layers):     # the committed tokens, bit for bit
            a, b_ = ref.Cache(got[l], D), ref.Cache(s.pages[l], D)
            for b in range(len(lens)):
                for p in range(int(want[b])):
                    for h in range(H):
                        for x, y in zip(a.get(s.table[b, p // P], h, p % P),
                                        b_.get(s.table[b, p // P], h, p % P)):
                            assert np.array_equal(x, y)
        others = np.setdiff1d(np.arange(s.pages.shape[1]), s.table[s.table >= 0])
        assert np.array_equal(got[:, others], s.pages[:, others])


def test_commit_errors_leave_the_sequence(gpu_lib):
    t = torch()
    rng = np.random.default_rng(21)
    s = Setup(rng, [40, 40, 10, 40], 1, 64, 32, layers=2)
    s.gpu()
    before = s.g_pages.clone()
    N = 12
    parent = rand_trees(rng, 4, N)
    for accept, change, code in (([N, -1, 0, 0], None, gpu_lib.GDN_ERR_ACCEPT_RANGE),
                                 ([0, 0, 3, 0], None, gpu_lib.GDN_ERR_ROW_RANGE),
                                 ([0, 0, 0, 3], (3, 5, 7), gpu_lib.GDN_ERR_BAD_TREE)):
        par = parent.copy()
        if change:
            par[change[0], change[1]] = change[2]
        s.status.zero_()
        lens = s.g_len.clone()
        if code != gpu_lib.GDN_ERR_ROW_RANGE:
            lens[2] = 40
            s.g_table[2] = s.g_table[0]
        out = t.zeros_like(lens)
        gpu_lib.gdn_kv4_commit(s.g_pages, s.g_table, lens, i32(accept), out, N=N,
                               parent=i32(par), status=s.status)
        assert int(s.status.item()) == code
        for b in range(4):
            failed = (accept[b] not in range(N)) or (int(lens[b]) < N) or bool(change and
                                                                             b == change[0])
            assert int(out[b]) == (int(lens[b]) if failed else
                                   int(lens[b]) - N + len(ref.path_of(parent[b], accept[b])))
    assert t.equal(s.g_pages, before)     # accepted roots move nothing


# ------------------------------------------------------------------ pool
def test_pool_random_walk(gpu_lib):
    """Release, fork and reserve in random order against the plain pool."""
    t, rng = torch(), np.random.default_rng(30)
    P, n_pages, rows, width, layers, H, D = 64, 61, 14, 6, 2, 2, 64
    pages = rng.integers(0, 256, (layers, n_pages, H, P // 32, 36 * D), dtype=np.uint8)
    pool = ref.Pool(np.full((rows, width), -1), np.zeros(rows, np.int64),
                    np.zeros(n_pages, np.int64), P, pages)
    g = [i32(pool.table), i32(pool.kv_len), i32(pool.ref)]
    g_pages, status = cuda(pages), status_word()
    refused = 0
    for step in range(120):
        F = int(rng.integers(1, 6))
        pick = rng.permutation(rows)[:F]
        kind = rng.integers(0, 4)
        status.zero_()
        if kind == 0:
            keep = np.where(rng.random(F) < 0.5, 0, rng.integers(0, P * width, F))
            pool.release(pick, keep)
            gpu_lib.gdn_kv4_release(*g, i32(pick), i32(keep), page_tokens=P, status=status)
        elif kind == 1:
            empty = [r for r in range(rows) if pool.kv_len[r] == 0][:F]
            full = [r for r in range(rows) if r not in empty]
            if not empty or not full:
                continue
            src = rng.choice(full, len(empty))
            pool.fork(src, empty)
            gpu_lib.gdn_kv4_fork(*g, i32(src), i32(empty), page_tokens=P, status=status)
        else:
            new = np.minimum(pool.kv_len[pick] + rng.integers(0, 150, F), P * width)
            failed = pool.reserve(pick, new)
            refused += len(failed) > 0
            ws = t.empty(gpu_lib.gdn_kv4_reserve_workspace_bytes(F), dtype=t.uint8, device="cuda")
            gpu_lib.gdn_kv4_reserve(g_pages, *g, i32(pick), i32(new), ws, status=status)
            assert int(status.item()) == (gpu_lib.GDN_ERR_POOL_EMPTY if failed else 0)
        for got, want in zip(g, (pool.table, pool.kv_len, pool.ref)):
            assert np.array_equal(got.cpu().numpy(), want)
        held = np.bincount(pool.table[pool.table >= 0].ravel(), minlength=n_pages)
        assert np.array_equal(held, pool.ref)
    assert np.array_equal(g_pages.cpu().numpy(), pages)
    assert refused > 0


def test_pool_many_rows_and_pages(gpu_lib):
    """More rows and pages than one pass of a block takes."""
    t, rng = torch(), np.random.default_rng(31)
    P, n_pages, rows, width = 32, 20000, 2500, 8
    pool = ref.Pool(np.full((rows, width), -1), np.zeros(rows, np.int64),
                    (rng.random(n_pages) < 0.3).astype(np.int64), P)
    g = [i32(pool.table), i32(pool.kv_len), i32(pool.ref)]
    pages = t.zeros(1, n_pages, 1, 1, 36 * 64, dtype=t.uint8, device="cuda")
    order, new = rng.permutation(rows), rng.integers(0, P * width + 1, rows)
    ws = t.empty(gpu_lib.gdn_kv4_reserve_workspace_bytes(rows), dtype=t.uint8, device="cuda")
    status = status_word()
    gpu_lib.gdn_kv4_reserve(pages, *g, i32(order), i32(new), ws, status=status)
    assert pool.reserve(order, new) == [] and int(status.item()) == 0
    gpu_lib.gdn_kv4_release(*g, i32(order[:1500]), i32(new[:1500] // 2), page_tokens=P,
                            status=status)
    pool.release(order[:1500], new[:1500] // 2)
    for got, want in zip(g, (pool.table, pool.kv_len, pool.ref)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_pool_refusals(gpu_lib):
    """Rows out of range, branches onto rows in use, shrinking reserves: left and reported."""
    t = torch()
    P = 32
    table, kv_len, count = i32([[0, 1], [2, -1], [-1, -1]]), i32([40, 5, 0]), i32([1, 1, 1, 0])
    pages = t.zeros(1, 4, 1, 1, 36 * 64, dtype=t.uint8, device="cuda")
    before = [x.clone() for x in (table, kv_len, count)]
    ws = t.empty(64, dtype=t.uint8, device="cuda")
    status = status_word()
    for call in (
            lambda: gpu_lib.gdn_kv4_release(table, kv_len, count, i32([3]), i32([0]),
                                            page_tokens=P, status=status),
            lambda: gpu_lib.gdn_kv4_release(table, kv_len, count, i32([0]), i32([-1]),
                                            page_tokens=P, status=status),
            lambda: gpu_lib.gdn_kv4_fork(table, kv_len, count, i32([0]), i32([1]), page_tokens=P,
                                         status=status),
            lambda: gpu_lib.gdn_kv4_fork(table, kv_len, count, i32([-1]), i32([2]), page_tokens=P,
                                         status=status),
            lambda: gpu_lib.gdn_kv4_reserve(pages, table, kv_len, count, i32([0]), i32([39]), ws,
                                            status=status),
            lambda: gpu_lib.gdn_kv4_reserve(pages, table, kv_len, count, i32([0]), i32([65]), ws,
                                            status=status)):
        status.zero_()
        call()
        assert int(status.item()) == gpu_lib.GDN_ERR_ROW_RANGE
        assert all(t.equal(x, y) for x, y in zip((table, kv_len, count), before))


# ------------------------------------------------------------------ streams and graphs
def test_attention_in_a_graph_follows_the_lengths(gpu_lib):
    """A captured append + attention replayed with other lengths equals fresh calls."""
    rng, t = np.random.default_rng(40), torch()
    s = Setup(rng, [300, 40, 700], 2, 128, 64, slack=40)
    s.fill(rng)
    kw = s.gpu()
    q = t.from_numpy(rng.standard_normal((3, 4, 8, 128))).cuda().to(t.bfloat16)
    k = t.from_numpy(rng.standard_normal((3, 4, 2, 128))).cuda().to(t.bfloat16)
    o = t.empty_like(q)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(3, 4, 8, 2, 128), dtype=t.uint8,
                 device="cuda")

    def step(out, stream=None):
        gpu_lib.gdn_kv4_append(k, k, s.g_pages, s.g_table, s.g_len, stream=stream, **kw)
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, out, ws, scale=0.09,
                                  stream=stream, **kw)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    step(o, side)
    side.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=side):
        step(o)
    for lens in ([304, 44, 704], [308, 3, 0], [20, 48, 708]):   # written positions only
        s.g_len.copy_(i32(lens))
        t.cuda.synchronize()
        o.fill_(9)
        g.replay()
        t.cuda.synchronize()
        fresh = t.empty_like(q)
        step(fresh)
        assert t.equal(o, fresh)
    assert int(s.status.item()) == 0


def test_lengths_rewritten_on_the_stream_between_calls(gpu_lib):
    """Calls issued back to back, each after a kernel that rewrites the lengths, each
    follow theirs (the run of a block is worked out early, and again on a change)."""
    rng, t = np.random.default_rng(41), torch()
    s = Setup(rng, [3000, 2500], 2, 128, 64)
    kw = s.gpu()
    x = t.randn(2, 3000, 2, 128, device="cuda")
    gpu_lib.gdn_kv4_append(x, x, s.g_pages, s.g_table, s.g_len, **kw)
    q = t.randn(2, 1, 8, 128, device="cuda").to(t.bfloat16)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(2, 1, 8, 2, 128), dtype=t.uint8,
                 device="cuda")
    plans = [i32([3000 - 311 * i, 1 + 350 * i]) for i in range(8)]
    outs = [t.empty_like(q) for _ in plans]
    t.cuda.synchronize()
    for plan, o in zip(plans, outs):
        s.g_len.copy_(plan)
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.09, **kw)
    t.cuda.synchronize()
    for plan, o in zip(plans, outs):
        s.g_len.copy_(plan)
        t.cuda.synchronize()
        alone = t.empty_like(q)
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, alone, ws, scale=0.09, **kw)
        t.cuda.synchronize()
        assert t.equal(o, alone)
    assert int(s.status.item()) == 0


def test_more_sequences_than_are_kept(gpu_lib):
    """Over a thousand sequences (lengths looked up instead of kept), some empty, with trees."""
    rng, t = np.random.default_rng(42), torch()
    B, N = 1100, 3
    lens = [int(n) for n in rng.integers(0, 90, B)]
    s = Setup(rng, lens, 1, 64, 32)
    kw = s.gpu()
    x = t.randn(B, 90, 1, 64, device="cuda")
    gpu_lib.gdn_kv4_append(x, -x, s.g_pages, s.g_table, s.g_len, **kw)
    q = t.randn(B, N, 2, 64, device="cuda").to(t.bfloat16)
    parent = i32(np.tile([-1, 0, 0], (B, 1)))
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(B, N, 2, 1, 64), dtype=t.uint8,
                 device="cuda")
    o, one = t.full_like(q, 3), t.full_like(q, 3)
    gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.1, parent=parent,
                              **kw)
    for b in range(0, B, 100):    # in pieces
        n = min(100, B - b)
        gpu_lib.gdn_kv4_attention(q[b:b + n], s.g_pages, s.g_table[b:b + n], s.g_len[b:b + n],
                                  one[b:b + n], ws, scale=0.1, parent=parent[b:b + n], **kw)
    assert int(s.status.item()) == 0
    # other runs, other orders of the sums: equal up to the probabilities' rounding
    assert bool(((o.float() - one.float()).abs() <= 2.0 ** -7 * one.float().abs() + 2.0 ** -8).all())
    assert not o[[b for b in range(B) if lens[b] == 0]].any()
    bad = parent.clone()
    bad[1050, 1] = 7
    gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.1, parent=bad, **kw)
    assert int(s.status.item()) == (gpu_lib.GDN_ERR_BAD_TREE if lens[1050] else 0)


def test_parents_rewritten_on_the_stream_between_calls(gpu_lib):
    """The same for the trees: a malformed one between two good ones, back to back."""
    rng, t = np.random.default_rng(43), torch()
    s = Setup(rng, [900, 700], 2, 128, 64)
    kw = s.gpu()
    x = t.randn(2, 900, 2, 128, device="cuda")
    gpu_lib.gdn_kv4_append(x, x, s.g_pages, s.g_table, s.g_len, **kw)
    N = 22
    q = t.randn(2, N, 4, 128, device="cuda").to(t.bfloat16)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(2, N, 4, 2, 128), dtype=t.uint8,
                 device="cuda")
    plans = [i32(rand_trees(rng, 2, N)) for _ in range(6)]
    plans[2][1, 5] = 9
    outs, parent = [t.empty_like(q) for _ in plans], plans[-1].clone()
    t.cuda.synchronize()
    for plan, o in zip(plans, outs):
        parent.copy_(plan)
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.09,
                                  parent=parent, **kw)
    t.cuda.synchronize()
    assert int(s.status.item()) == gpu_lib.GDN_ERR_BAD_TREE
    for plan, o in zip(plans, outs):
        alone = t.empty_like(q)
        t.cuda.synchronize()
        gpu_lib.gdn_kv4_attention(q, s.g_pages, s.g_table, s.g_len, alone, ws, scale=0.09,
                                  parent=plan, **kw)
        t.cuda.synchronize()
        assert t.equal(o, alone)
    assert not outs[2][1].any() and outs[2][0].any()


@pytest.mark.parametrize("n_pages, F, offset, short", [
    (4095, 1, 0, False), (4096, 40, 1, False), (8193, 40, 0, True), (20011, 1300, 3, False),
    (20011, 1300, 0, True), (7, 2, 1, False), (3100, 1024, 0, True)])
def test_reserve_of_large_pools(gpu_lib, n_pages, F, offset, short):
    """Pools over several reads of the counts, counts at any 4-byte address, more rows
    than one pass takes, too few pages: as the plain pool."""
    rng, t = np.random.default_rng(n_pages + F + offset), torch()
    P, width = 32, 3
    table, kv_len = np.full((F, width), -1, np.int64), np.zeros(F, np.int64)
    want = rng.integers(1, width * P + 1, F)
    need = int((-(-want // P)).sum())
    held = rng.permutation(n_pages)[:n_pages - (need - 2 if short else min(n_pages, need + 1))]
    count = np.zeros(n_pages, np.int64)
    count[held] = rng.integers(1, 4, len(held))
    room = t.zeros(n_pages + offset, dtype=t.int32, device="cuda")
    room[offset:] = i32(count)
    g = (i32(table), i32(kv_len), room[offset:])
    pages = t.zeros(n_pages, 1, 1, 36 * 64, dtype=t.uint8, device="cuda")
    status = status_word()
    ws = t.empty(gpu_lib.gdn_kv4_reserve_workspace_bytes(F), dtype=t.uint8, device="cuda")
    order = [int(r) for r in rng.permutation(F)]
    new = [int(want[r]) for r in order]
    pool = ref.Pool(table, kv_len, count, P)
    failed = pool.reserve(order, new)
    gpu_lib.gdn_kv4_reserve(pages, *g, i32(order), i32(new), ws, status=status)
    for got, exp in zip(g, (table, kv_len, count)):
        assert np.array_equal(got.cpu().numpy(), exp)
    assert bool(failed) == short
    assert int(status.item()) == (gpu_lib.GDN_ERR_POOL_EMPTY if short else 0)


# ------------------------------------------------------------------ wide tiles' scale
@pytest.mark.parametrize("dtype, spread, D", [
    ("bf16", 8, 128), ("f16", 8, 64), ("bf16", 9, 256), ("bf16", 60, 128), ("f16", 20, 256)])
def test_attention_rows_of_many_magnitudes_in_a_wide_tile(gpu_lib, dtype, spread, D):
    """80 rows whose largest magnitudes span 2^spread (up to 2^8 they share a scale), with
    elements over the type's whole precision and some rows of zeros."""
    rng, t = np.random.default_rng(50 + spread + D), torch()
    s = Setup(rng, [333, 150], 1, D, 64)
    cache = s.fill(rng)
    B, N, Hq = 2, 20, 4
    q = rng.uniform(-1, 1, (B, N, Hq, D)) * 2.0 ** rng.integers(-14, 1, (B, N, Hq, D))
    row = rng.integers(0, spread + 1, (B, N, Hq))
    row[:, 0, 0], row[:, 1, 0] = 0, spread
    top = np.abs(q).max(-1)
    q = q / 2.0 ** np.floor(np.log2(top))[..., None] * 2.0 ** (4.0 - row)[..., None]
    q[:, 5, 1] = 0
    q = t.from_numpy(q).cuda().to(tdtype(dtype))
    check_attention(gpu_lib, s, cache, q, dtype, 0.05)
    check_attention(gpu_lib, s, cache, q, dtype, 0.05, rand_trees(rng, B, N))


def test_attention_infinite_and_nan_queries_in_a_wide_tile(gpu_lib):
    """They stay in their row: the others' bits are those beside rows of zeros."""
    rng, t = np.random.default_rng(60), torch()
    s = Setup(rng, [500], 1, 128, 32)
    s.fill(rng)
    kw = s.gpu()
    q = t.from_numpy(rng.standard_normal((1, 24, 4, 128))).cuda().to(t.bfloat16)
    ws = t.empty(gpu_lib.gdn_kv4_attention_workspace_bytes(1, 24, 4, 1, 128), dtype=t.uint8,
                 device="cuda")

    def run(value):
        x, o = q.clone(), t.empty_like(q)
        x[0, 3, 1, 7], x[0, 9, 0] = value, value
        gpu_lib.gdn_kv4_attention(x, s.g_pages, s.g_table, s.g_len, o, ws, scale=0.1, **kw)
        return o

    x = q.clone()
    x[0, 3, 1], x[0, 9, 0] = 0, 0
    base = t.empty_like(q)
    gpu_lib.gdn_kv4_attention(x, s.g_pages, s.g_table, s.g_len, base, ws, scale=0.1, **kw)
    others = t.ones(1, 24, 4, dtype=t.bool, device="cuda")
    others[0, 3, 1] = others[0, 9, 0] = False
    for value in (float("nan"), float("inf"), -float("inf")):
        o = run(value)
        assert t.equal(o[others], base[others])
        assert not t.isfinite(o[0, 9, 0]).any()
    assert int(s.status.item()) == 0
