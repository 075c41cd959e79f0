"""Rotary append to the 4-bit cache on the GPU: bit for bit what turning, rounding and quantising
give one after another."""
import numpy as np
import pytest

import kv4_forms_reference as forms
import kv4_reference as ref
from gpu_helpers import torch
from test_gpu_kv4 import Setup, cuda, i32, tdtype

pytestmark = pytest.mark.gpu


def angles(rng, n, pairs):
    a = np.arange(n)[:, None] * rng.uniform(0.001, 1, pairs)
    return np.stack((np.cos(a), np.sin(a)), 1).astype(np.float32)


def block(rng, B, N, Hq, H, D, dtype):
    """q, k, v as slices of one fused projection."""
    t = torch()
    qkv = t.from_numpy(rng.standard_normal((B, N, (Hq + 2 * H) * D))).cuda().to(tdtype(dtype))
    return [x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, H * D, H * D], -1)]


def as_float(x):
    return x.float().cpu().numpy()


def expect(s, q, k, v, pos, cs, axis, adjacent, dtype):
    """q_out of the reference; its pages are appended to s.pages."""
    N = q.shape[1]
    ref.append(ref.Cache(s.pages, s.D), s.table, s.lens, s.P,
               forms.turned(as_float(k), pos, cs, axis, adjacent), as_float(v), s.ks, s.vs)
    out = torch().from_numpy(forms.turned(as_float(q), pos, cs, axis, adjacent)).to(tdtype(dtype))
    for b, n in enumerate(s.lens):
        out[b, :max(0, N - max(0, int(n)))] = 0
    return out


CASES = [
    # dtype, lens, N, Hq, H, D, P, pairs, axes, adjacent
    ("bf16", [1], 1, 1, 1, 64, 32, 8, 1, False),
    ("bf16", [700], 1, 24, 4, 256, 64, 32, 3, False),
    ("f16", [33, 64, 31], 1, 8, 8, 128, 32, 64, 1, True),
    ("f32", [0, 5, 22, 23, 200], 22, 4, 2, 64, 96, 32, 3, False),   # absent nodes
    ("f32", [40, 16, 97], 16, 6, 2, 256, 64, 128, 2, True),         # all channels
    ("bf16", [300], 300, 3, 1, 256, 64, 40, 3, False),              # a prompt, odd pairs
    ("bf16", [161, 130], 65, 6, 3, 128, 32, 24, 4, True),
    ("f16", [64], 32, 34, 2, 64, 1664, 16, 3, False),
    ("bf16", [130], 129, 1, 1, 64, 32, 32, 1, False),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype, lens, N, Hq, H, D, P, pairs, axes, adjacent", CASES)
def test_append_rotary(gpu_lib, dtype, lens, N, Hq, H, D, P, pairs, axes, adjacent, in_place):
    rng, t = np.random.default_rng(N * D + pairs), torch()
    s = Setup(rng, lens, H, D, P)
    kw = s.gpu()
    B = len(lens)
    q, k, v = block(rng, B, N, Hq, H, D, dtype)
    pos = rng.integers(0, 500, (axes, B, N))
    for b, n in enumerate(lens):   # not looked at
        pos[:, b, :max(0, N - n)] = -12345
    cs = angles(rng, 500, pairs)
    axis = None if axes == 1 else rng.integers(0, axes, pairs).astype(np.uint8)
    want = expect(s, q, k, v, pos, cs, axis, adjacent, dtype)
    kept = [k.clone(), v.clone(), q.clone()]
    # apart: with strides of its own, between guards
    room = t.full((B, N, Hq + 2, D), 7.0, dtype=q.dtype, device="cuda")
    out = q if in_place else room[:, :, 1:Hq + 1]
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), cuda(cs), s.g_pages, s.g_table, s.g_len, out,
                                  axis=None if axis is None else cuda(axis), adjacent=adjacent,
                                  **kw)
    assert int(s.status.item()) == 0
    assert t.equal(out.cpu(), want)
    assert np.array_equal(s.g_pages.cpu().numpy(), s.pages)
    assert t.equal(k, kept[0]) and t.equal(v, kept[1])
    if not in_place:
        assert t.equal(q, kept[2]) and (room[:, :, 0] == 7).all() and (room[:, :, -1] == 7).all()


def test_positions_as_a_slice(gpu_lib):
    """Positions with strides between axes and sequences, the table longer than it is used."""
    rng, t = np.random.default_rng(2), torch()
    s = Setup(rng, [20, 40, 50], 2, 64, 32)
    kw = s.gpu()
    q, k, v = block(rng, 3, 5, 4, 2, 64, "bf16")
    big = rng.integers(0, 64, (6, 4, 9))
    cs, axis = angles(rng, 64, 16), rng.integers(0, 3, 16).astype(np.uint8)
    pos = big[::2, 1:, 2:7]
    want = expect(s, q, k, v, pos, cs, axis, False, "bf16")
    out = t.empty(q.shape, dtype=q.dtype, device="cuda")
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(big)[::2, 1:, 2:7], cuda(cs), s.g_pages, s.g_table,
                                  s.g_len, out, axis=cuda(axis), **kw)
    assert t.equal(out.cpu(), want) and np.array_equal(s.g_pages.cpu().numpy(), s.pages)


@pytest.mark.parametrize("bad", ["low", "high", "axis"])
def test_bad_positions_leave_their_pairs_and_are_reported(gpu_lib, bad):
    rng, t = np.random.default_rng(3), torch()
    s = Setup(rng, [9, 40], 1, 128, 32)
    kw = s.gpu()
    q, k, v = block(rng, 2, 4, 2, 1, 128, "f16")
    pos = rng.integers(0, 30, (2, 2, 4))
    axis = rng.integers(0, 2, 32).astype(np.uint8)
    if bad == "axis":
        axis[5] = 2
    else:
        pos[1, 0, 2] = -1 if bad == "low" else 30
    cs = angles(rng, 30, 32)
    want = expect(s, q, k, v, pos, cs, axis, False, "f16")
    out = t.empty(q.shape, dtype=q.dtype, device="cuda")
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), cuda(cs), s.g_pages, s.g_table, s.g_len, out,
                                  axis=cuda(axis), **kw)
    assert int(s.status.item()) == gpu_lib.GDN_ERR_POSITION_RANGE
    assert t.equal(out.cpu(), want) and np.array_equal(s.g_pages.cpu().numpy(), s.pages)


def test_refused_rows_and_bad_pages(gpu_lib):
    """A length of -1 (a row that found no page) writes nothing and gives q_out = 0; a bad page
    number leaves out its keys only."""
    rng, t = np.random.default_rng(4), torch()
    s = Setup(rng, [60, 60, 60], 2, 64, 32)
    kw = s.gpu()
    q, k, v = block(rng, 3, 4, 4, 2, 64, "bf16")
    pos, cs = rng.integers(0, 30, (1, 3, 4)), angles(rng, 30, 16)
    out = t.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    for row, code in ((0, gpu_lib.GDN_ERR_ROW_RANGE), (1, gpu_lib.GDN_ERR_PAGE_RANGE)):
        s.g_pages.copy_(cuda(s.pages))
        s.g_len.copy_(i32(s.lens))
        s.status.zero_()
        before = s.pages.copy()
        table, lens = s.table.copy(), s.lens.copy()
        if row == 0:
            s.g_len[0] = -1
            s.lens[0] = 0
        else:
            s.g_table[1, 1] = 1 << 20
            s.lens[1] = 0      # (the reference's row appends nothing)
        want = expect(s, q, k, v, pos, cs, None, False, "bf16")
        if row == 1:
            lens1 = np.array([60, 60, 60])
            want[1] = t.from_numpy(forms.turned(as_float(q), pos, cs, None, False))[1].to(q.dtype)
        gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), cuda(cs), s.g_pages, s.g_table, s.g_len,
                                      out, **kw)
        assert int(s.status.item()) == code
        assert t.equal(out.cpu(), want) and np.array_equal(s.g_pages.cpu().numpy(), s.pages)
        s.pages, s.table, s.lens = before, table, lens


def test_nan_and_infinity_stay_in_their_pairs(gpu_lib):
    """A NaN key makes its pair NaN, which the cache stores as 0 and reports; queries keep theirs."""
    rng, t = np.random.default_rng(5), torch()
    s = Setup(rng, [40], 1, 64, 32, ones=True)
    kw = s.gpu()
    q, k, v = (x.contiguous() for x in block(rng, 1, 2, 1, 1, 64, "f32"))
    k[0, 0, 0, 3] = float("nan")
    q[0, 1, 0, 20] = float("inf")
    q[0, 1, 0, 50] = float("nan")
    pos, cs = np.array([[[3, 4]]]), angles(rng, 30, 16)
    want = expect(s, q, k, v, pos, cs, None, False, "f32")
    out = t.empty_like(q)
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), cuda(cs), s.g_pages, s.g_table, s.g_len, out,
                                  **kw)
    assert int(s.status.item()) == gpu_lib.GDN_ERR_NONFINITE
    assert t.equal(out.isnan().cpu(), want.isnan())
    assert t.equal(out.nan_to_num(0.0).cpu(), want.nan_to_num(0.0))
    assert np.array_equal(s.g_pages.cpu().numpy(), s.pages)


def test_unturned_is_append(gpu_lib):
    """Positions whose angle is 0 give gdn_kv4_append's bytes and the queries themselves."""
    rng, t = np.random.default_rng(6), torch()
    s = Setup(rng, [70, 33], 2, 128, 32)
    kw = s.gpu()
    q, k, v = block(rng, 2, 20, 4, 2, 128, "bf16")
    cs = t.zeros(1, 2, 64, device="cuda")
    cs[:, 0] = 1
    other = s.g_pages.clone()
    out = t.empty(q.shape, dtype=q.dtype, device="cuda")
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(np.zeros((1, 2, 20))), cs, s.g_pages, s.g_table,
                                  s.g_len, out, **kw)
    gpu_lib.gdn_kv4_append(k, v, other, s.g_table, s.g_len, **kw)
    assert t.equal(s.g_pages, other) and t.equal(out, q)


def test_in_a_graph_on_a_stream(gpu_lib):
    """A captured call follows the lengths and positions that the buffers hold at replay."""
    rng, t = np.random.default_rng(7), torch()
    s = Setup(rng, [40, 70], 2, 128, 32, slack=40)
    kw = s.gpu()
    q, k, v = block(rng, 2, 3, 4, 2, 128, "bf16")
    pos, cs = rng.integers(0, 60, (1, 2, 3)), angles(rng, 90, 32)
    g_pos, g_cs = i32(pos), cuda(cs)
    out = t.empty(q.shape, dtype=q.dtype, device="cuda")
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        call = gpu_lib.bind_kv4_append_rotary(q, k, v, g_pos, g_cs, s.g_pages, s.g_table, s.g_len,
                                              out, **kw)
        call()
        side.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            call()
    want = expect(s, q, k, v, pos, cs, None, False, "bf16")
    for step in range(1, 3):
        s.g_len += 3
        g_pos += 3
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        s.lens = s.lens + 3
        want = expect(s, q, k, v, pos + 3 * step, cs, None, False, "bf16")
    assert t.equal(out.cpu(), want) and np.array_equal(s.g_pages.cpu().numpy(), s.pages)


def test_empty_batch(gpu_lib):
    t = torch()
    e = lambda *n, dt=t.bfloat16: t.empty(n, dtype=dt, device="cuda")  # noqa: E731
    gpu_lib.gdn_kv4_append_rotary(e(0, 3, 4, 64), e(0, 3, 2, 64), e(0, 3, 2, 64),
                                  e(1, 0, 3, dt=t.int32), e(9, 2, 16, dt=t.float32),
                                  e(4, 2, 1, 36 * 64, dt=t.uint8), e(0, 2, dt=t.int32),
                                  e(0, dt=t.int32), e(0, 3, 4, 64))
