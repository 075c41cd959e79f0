"""Rotary append on the GPU: pairs without a position pass as they are.  A turn by 0 would not do:
0 times an infinity or a NaN is no number, and -0 + 0 is 0."""
import numpy as np
import pytest

import kv4_forms_reference as forms
import kv4_reference as ref
from gpu_helpers import torch
from test_gpu_kv4 import Setup, cuda, i32
from test_gpu_kv4_rotary import angles, as_float, block

pytestmark = pytest.mark.gpu

ODD = [np.inf, -np.inf, np.nan, -0.0, 0.0]


def passing(x, positions, n_positions, axis, pairs, adjacent):
    """Channels [B,N,1,D] of pairs without a position, and channels that are in no pair."""
    B, N, _, D = x.shape
    out = np.ones((B, N, 1, D), bool)
    for b in range(B):
        for n in range(N):
            for i in range(pairs):
                a = 0 if axis is None else int(axis[i])
                there = a < positions.shape[0] and 0 <= positions[a, b, n] < n_positions
                for ch in (2 * i, 2 * i + 1) if adjacent else (i, i + pairs):
                    out[b, n, 0, ch] = not there
    return out


def turned(x, positions, cs, axis, adjacent):
    stays = passing(x, positions, cs.shape[0], axis, cs.shape[2], adjacent)
    return np.where(stays, x, forms.turned(x, positions, cs, axis, adjacent))


def same_bits(got, want):
    """The same values, signs of zeros among them; a NaN is a NaN."""
    t = torch()
    n = t.int32 if got.dtype == t.float32 else t.int16
    nan = got.isnan()
    return t.equal(nan, want.isnan()) and t.equal(got.view(n)[~nan], want.view(n)[~nan])


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype, H, D, pairs, N", [("bf16", 1, 64, 32, 4), ("f16", 2, 128, 24, 3),
                                                   ("f32", 1, 256, 128, 5), ("bf16", 2, 256, 32, 40)])
def test_pairs_without_a_position(gpu_lib, dtype, H, D, pairs, N, in_place, adjacent):
    rng, t = np.random.default_rng(N * D + pairs + adjacent), torch()
    lens = [N + 7, N, 70]
    s = Setup(rng, lens, H, D, 32)
    kw = s.gpu()
    q, k, v = block(rng, 3, N, 2 * H, H, D, dtype)
    # zeros, infinities and NaN in a sixteenth of the channels
    for x in (q, k):
        at = t.from_numpy(rng.random(x.shape) < 1 / 16).cuda()
        odd = t.from_numpy(rng.choice(ODD, x.shape)).cuda().to(x.dtype)
        x.copy_(t.where(at, odd, x))
    axis = rng.integers(0, 4, pairs).astype(np.uint8)     # the last of them is none
    pos = rng.integers(-3, 33, (3, 3, N))                 # some lie outside
    cs = angles(rng, 30, pairs)
    args = (pos, cs, axis, adjacent)
    with np.errstate(invalid="ignore"):
        ref.append(ref.Cache(s.pages, D), s.table, s.lens, 32, turned(as_float(k), *args),
                   as_float(v), s.ks, s.vs)
        want = t.from_numpy(turned(as_float(q), *args)).to(q.dtype)
    out = q if in_place else t.empty(q.shape, dtype=q.dtype, device="cuda")
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), cuda(cs), s.g_pages, s.g_table, s.g_len, out,
                                  axis=cuda(axis), adjacent=adjacent, **kw)
    assert int(s.status.item()) in (gpu_lib.GDN_ERR_POSITION_RANGE, gpu_lib.GDN_ERR_NONFINITE)
    assert same_bits(out.cpu(), want)
    assert np.array_equal(s.g_pages.cpu().numpy(), s.pages)


def test_a_finite_key_beside_an_infinity_stays(gpu_lib):
    """One pair, no position: the infinity is stored saturated, its partner as it is, and a zero
    keeps its sign; nothing else is reported than the position and the infinity."""
    rng, t = np.random.default_rng(9), torch()
    s = Setup(rng, [1], 1, 64, 32, ones=True)
    kw = s.gpu()
    q = t.zeros(1, 1, 1, 64, device="cuda")
    k, v = t.ones_like(q), t.ones_like(q)
    k[..., 3], q[..., 3] = float("inf"), float("inf")     # pair 3: channels 3 and 35
    q[..., 35], q[..., 4], q[..., 36] = 1.5, -0.0, -2.0
    kept = q.clone()
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32([[[-1]]]), cuda(angles(rng, 4, 32)), s.g_pages,
                                  s.g_table, s.g_len, q, **kw)
    assert same_bits(q.cpu(), kept.cpu())
    ko, vo = t.empty_like(q), t.empty_like(q)
    gpu_lib.gdn_kv4_read(s.g_pages, s.g_table, s.g_len, ko, vo, **kw)
    # (elsewhere 1 is stored as 6 * 11/64: 1/6 lies between 10/64 and 11/64, next to the latter)
    assert ko[0, 0, 0, 3] == 2688 and (ko[0, 0, 0, 16:] == 6 * 11 / 64).all()


@pytest.mark.parametrize("B, N", [(1, 3), (3, 1), (1, 1)])
def test_in_place_with_another_stride_of_an_axis_of_one(gpu_lib, B, N):
    rng, t = np.random.default_rng(B + 4 * N), torch()
    s = Setup(rng, [40, 21, 33][:B], 2, 64, 32)
    kw = s.gpu()
    q, k, v = (x.contiguous() for x in block(rng, B, N, 4, 2, 64, "bf16"))
    pos, cs = rng.integers(0, 30, (1, B, N)), angles(rng, 30, 16)
    want = t.from_numpy(forms.turned(as_float(q), pos, cs, None, False)).to(q.dtype)
    strides = (8 if B == 1 else q.stride(0), 16 if N == 1 else q.stride(1), 64, 1)
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), cuda(cs), s.g_pages, s.g_table, s.g_len,
                                  q.as_strided(q.shape, strides), **kw)
    assert int(s.status.item()) == 0 and t.equal(q.cpu(), want)


def test_nodes_outermost(gpu_lib):
    """q_out with the sequences of a node beside each other, rows one after another."""
    rng, t = np.random.default_rng(10), torch()
    s = Setup(rng, [40, 21, 33], 2, 64, 32)
    kw = s.gpu()
    q, k, v = block(rng, 3, 5, 4, 2, 64, "f16")
    pos, cs = rng.integers(0, 30, (1, 3, 5)), angles(rng, 30, 32)
    want = t.from_numpy(forms.turned(as_float(q), pos, cs, None, True)).to(q.dtype)
    out = t.empty(5, 3, 4, 64, dtype=q.dtype, device="cuda").transpose(0, 1)
    gpu_lib.gdn_kv4_append_rotary(q, k, v, i32(pos), cuda(cs), s.g_pages, s.g_table, s.g_len, out,
                                  adjacent=True, **kw)
    assert int(s.status.item()) == 0 and t.equal(out.cpu(), want)
