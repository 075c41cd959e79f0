"""CPU checks of the rotary append and of the windowed and shared forms of the attention: struct
layout, refusals of the C ABI and of the binding (none of these calls reaches the GPU), and the
reference's own definitions."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import hybrid_gated_deltanet_delta_gb300 as gdn
import kv4_forms_reference as forms
import kv4_reference as ref
from test_kv4_host import CACHE_CHECKS, _cache, lib  # noqa: F401

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
V = ctypes.c_void_p


def test_rotary_struct_layout_matches_c(tmp_path):
    fields = [f for f, _ in gdn.Rotary._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include "gdn.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void){'
                   'printf("%zu", sizeof(gdn_rotary));'
                   + "".join(f'printf(" %zu", offsetof(gdn_rotary, {f}));' for f in fields)
                   + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", INCLUDE, str(src), "-o", str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    assert got == [ctypes.sizeof(gdn.Rotary)] + [getattr(gdn.Rotary, f).offset for f in fields]


def _rotary(**kw):
    r = gdn.Rotary()
    base = dict(cos_sin=0x100, positions=0x200, pos_stride_axis=8, pos_stride_b=4,
                n_positions=100, n_axes=3, pairs=32, adjacent=0)
    base.update(kw)
    for key, val in base.items():
        setattr(r, key, val)
    return r


def append_rotary(lib, c, r, q=0x100, qsb=24576, qsn=6144, Hq=24, out=0x200, osb=24576, osn=6144,
                  k=0x300, v=0x400, dtype=gdn.GDN_BF16, ks=1024, N=4):
    return lib.gdn_kv4_append_rotary(ctypes.byref(c) if c else None, ctypes.byref(r) if r else None,
                                     V(q), qsb, qsn, Hq, V(out), osb, osn, V(k), V(v), dtype,
                                     4 * ks, ks, 4 * ks, ks, N, None)


@pytest.mark.parametrize("change, want", CACHE_CHECKS)
def test_cache_checks(lib, change, want):  # noqa: F811
    c = _cache(**change)
    assert append_rotary(lib, c, _rotary()) == want
    lead = (ctypes.byref(c), V(0x100), gdn.GDN_BF16, 4096, 1024, 4, 24, 1.0)
    trail = (V(0x200), None, V(0x300), 1 << 40, None)
    assert lib.gdn_kv4_attention_window(*lead, 4, 100, None, *trail) == want
    assert lib.gdn_kv4_attention_shared(*lead, None, V(0x400), 1, *trail) == want


@pytest.mark.parametrize("kw, rot, want", [
    (dict(N=0), {}, gdn.GDN_ERR_INVALID_ARG),
    (dict(N=(1 << 24) + 1), {}, gdn.GDN_ERR_UNSUPPORTED),
    (dict(dtype=3), {}, gdn.GDN_ERR_INVALID_ARG),
    (dict(Hq=0), {}, gdn.GDN_ERR_INVALID_ARG),
    (dict(Hq=22), {}, gdn.GDN_ERR_INVALID_ARG),
    (dict(Hq=65536), {}, gdn.GDN_ERR_UNSUPPORTED),
    (dict(q=0), {}, gdn.GDN_ERR_INVALID_ARG),
    (dict(out=0), {}, gdn.GDN_ERR_INVALID_ARG),
    (dict(k=0), {}, gdn.GDN_ERR_INVALID_ARG),
    (dict(v=0x404), {}, gdn.GDN_ERR_MISALIGNED),
    (dict(out=0x208), {}, gdn.GDN_ERR_MISALIGNED),
    (dict(qsn=6148), {}, gdn.GDN_ERR_MISALIGNED),
    (dict(osb=24572), {}, gdn.GDN_ERR_MISALIGNED),
    (dict(dtype=gdn.GDN_F32, qsn=6146), {}, gdn.GDN_ERR_MISALIGNED),
    (dict(out=0x100, osn=6152), {}, gdn.GDN_ERR_INVALID_ARG),      # in place, other strides
    ({}, dict(pairs=0), gdn.GDN_ERR_INVALID_ARG),
    ({}, dict(pairs=12), gdn.GDN_ERR_UNSUPPORTED),
    ({}, dict(pairs=136), gdn.GDN_ERR_UNSUPPORTED),
    ({}, dict(n_positions=0), gdn.GDN_ERR_INVALID_ARG),
    ({}, dict(n_axes=0), gdn.GDN_ERR_INVALID_ARG),
    ({}, dict(adjacent=2), gdn.GDN_ERR_INVALID_ARG),
    ({}, dict(cos_sin=0), gdn.GDN_ERR_INVALID_ARG),
    ({}, dict(cos_sin=0x104), gdn.GDN_ERR_MISALIGNED),
    ({}, dict(positions=0), gdn.GDN_ERR_INVALID_ARG),
    ({}, dict(positions=0x202), gdn.GDN_ERR_MISALIGNED),
])
def test_append_rotary_checks(lib, kw, rot, want):  # noqa: F811
    assert append_rotary(lib, _cache(), _rotary(**rot), **kw) == want


def test_append_rotary_without_structs(lib):  # noqa: F811
    assert append_rotary(lib, None, _rotary()) == gdn.GDN_ERR_INVALID_ARG
    assert append_rotary(lib, _cache(), None) == gdn.GDN_ERR_INVALID_ARG


ATTENTION = [
    (dict(Hq=22), gdn.GDN_ERR_INVALID_ARG),
    (dict(N=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(dtype=gdn.GDN_F32), gdn.GDN_ERR_UNSUPPORTED),
    (dict(dtype=9), gdn.GDN_ERR_INVALID_ARG),
    (dict(N=65, parent=0x400), gdn.GDN_ERR_UNSUPPORTED),
    (dict(q=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(o=0x204), gdn.GDN_ERR_MISALIGNED),
    (dict(sn=1028), gdn.GDN_ERR_MISALIGNED),
    (dict(lse=0x501), gdn.GDN_ERR_MISALIGNED),
    (dict(parent=0x402), gdn.GDN_ERR_MISALIGNED),
    (dict(ws=0), gdn.GDN_ERR_WORKSPACE),
    (dict(bytes=8), gdn.GDN_ERR_WORKSPACE),
    (dict(ws=0x308), gdn.GDN_ERR_MISALIGNED),
]
WINDOW = [(dict(window=0), gdn.GDN_ERR_INVALID_ARG), (dict(window=-5), gdn.GDN_ERR_INVALID_ARG),
          (dict(sinks=-1), gdn.GDN_ERR_INVALID_ARG)]
SHARED = [(dict(groups=0), gdn.GDN_ERR_INVALID_ARG), (dict(groups=3), gdn.GDN_ERR_INVALID_ARG),
          (dict(group=0), gdn.GDN_ERR_INVALID_ARG), (dict(group=0x602), gdn.GDN_ERR_MISALIGNED)]


def _attend(lib, form, kw):  # noqa: F811
    a = dict(N=4, Hq=24, dtype=gdn.GDN_BF16, q=0x100, o=0x200, sb=4096, sn=1024, parent=0, lse=0,
             ws=0x300, bytes=1 << 40, window=100, sinks=4, group=0x600, groups=2)
    a.update(kw)
    lead = (ctypes.byref(_cache()), V(a["q"]), a["dtype"], a["sb"], a["sn"], a["N"], a["Hq"], 1.0)
    trail = (V(a["o"]), V(a["lse"]), V(a["ws"]), a["bytes"], None)
    if form == "window":
        return lib.gdn_kv4_attention_window(*lead, a["sinks"], a["window"], V(a["parent"]), *trail)
    return lib.gdn_kv4_attention_shared(*lead, V(a["parent"]), V(a["group"]), a["groups"], *trail)


@pytest.mark.parametrize("kw, want", ATTENTION + WINDOW)
def test_window_checks(lib, kw, want):  # noqa: F811
    assert _attend(lib, "window", kw) == want


@pytest.mark.parametrize("kw, want", ATTENTION + SHARED)
def test_shared_checks(lib, kw, want):  # noqa: F811
    assert _attend(lib, "shared", kw) == want


def test_shared_workspace_sizes(lib):  # noqa: F811
    size = lib.gdn_kv4_attention_shared_workspace_bytes
    plain = lib.gdn_kv4_attention_workspace_bytes
    assert size(32, 1, 24, 4, 256, 1) >= 2 * 32 * 24 * 256 * 4
    assert size(32, 4, 24, 4, 256, 32) > size(32, 1, 24, 4, 256, 32) >= size(32, 1, 24, 4, 256, 1)
    assert size(32, 1, 24, 4, 256, 33) == 0 and size(32, 1, 24, 4, 256, 0) == 0
    assert size(0, 1, 24, 4, 256, 1) == 0 and size(8, 1, 25, 4, 256, 1) == 0
    assert size(8, 1, 24, 4, 80, 1) == 0
    assert size(8, 2048, 24, 4, 256, 2) == plain(8, 2048, 24, 4, 256)   # rows fill the tiles
    assert size(65535, 1 << 15, 4, 1, 64, 2) == 0                       # rows past 31 bits


def test_names_of_the_new_code(lib):  # noqa: F811
    assert gdn.status_string(gdn.GDN_ERR_POSITION_RANGE) == "GDN_ERR_POSITION_RANGE"


# ---- the binding
def _tensors(B=2, N=3, Hq=4, Hkv=2, D=64, pairs=16, axes=3):
    i32 = dict(dtype=torch.int32)
    return dict(q=torch.zeros(B, N, Hq, D), k=torch.zeros(B, N, Hkv, D), v=torch.zeros(B, N, Hkv, D),
                positions=torch.zeros(axes, B, N, **i32), cos_sin=torch.zeros(50, 2, pairs),
                pages=torch.zeros(4, Hkv, 1, 36 * D, dtype=torch.uint8),
                table=torch.zeros(B, 4, **i32), kv_len=torch.zeros(B, **i32),
                q_out=torch.zeros(B, N, Hq, D))


@pytest.mark.parametrize("kw, match", [
    (dict(v=torch.zeros(2, 3, 1, 64)), "share a shape"),
    (dict(q_out=torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)), "share a dtype"),
    (dict(q_out=torch.zeros(2, 2, 4, 64)), "share a shape"),
    (dict(cos_sin=torch.zeros(50, 32)), "cos_sin"),
    (dict(cos_sin=torch.zeros(50, 2, 16, dtype=torch.float64)), "cos_sin"),
    (dict(positions=torch.zeros(3, 2, 3)), "positions"),
    (dict(positions=torch.zeros(3, 2, 4, dtype=torch.int32)), "positions"),
    (dict(axis=torch.zeros(15, dtype=torch.uint8)), "axis"),
    (dict(axis=torch.zeros(16, dtype=torch.int32)), "axis"),
    (dict(), "current CUDA device"),               # tensors of the host
])
def test_binding_refuses_append_rotary(monkeypatch, kw, match):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a = _tensors()
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        gdn.gdn_kv4_append_rotary(**a)


def test_binding_refuses_attention(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a = _tensors()
    q = a["q"].to(torch.bfloat16)
    args = (q, a["pages"], a["table"], a["kv_len"])
    ws = torch.zeros(16, dtype=torch.uint8)
    group = torch.tensor([0, 2], dtype=torch.int32)
    for o, g, match in ((torch.zeros(2, 3, 4, 64), group, "q's shape and dtype"),
                        (torch.empty_like(q), group.long(), "group"),
                        (torch.empty_like(q), group, "current CUDA device")):
        with pytest.raises(ValueError, match=match):
            gdn.gdn_kv4_attention_shared(*args, g, o, ws, scale=1.0)
    with pytest.raises(ValueError, match="current CUDA device"):
        gdn.gdn_kv4_attention_window(*args, torch.empty_like(q), ws, scale=1.0, window=5)


# ---- the reference itself
def test_reference_rotation_is_a_rotation():
    """Lengths of pairs stay, positions add up: turning by p and then by r is turning by p + r."""
    rng = np.random.default_rng(0)
    angle = np.arange(40)[:, None] * rng.uniform(0.01, 1, 8)
    cs = np.stack((np.cos(angle), np.sin(angle)), 1).astype(np.float32)
    x = rng.standard_normal((1, 1, 2, 32)).astype(np.float32)

    def at(y, p, adjacent):
        return forms.turned(y, np.full((1, 1, 1), p), cs, None, adjacent)
    for adjacent in (False, True):
        twice, once = at(at(x, 11, adjacent), 17, adjacent), at(x, 28, adjacent)
        # two rotations of three roundings each, angles rounded once: 2^-24 of values below 8
        assert np.abs(twice - once).max() < 8 * 2.0 ** -20
        assert np.array_equal(once[..., 16:], x[..., 16:])
        assert abs((once ** 2).sum() - (x ** 2).sum()) < 1e-4
        assert not np.allclose(once[..., :16], x[..., :16], atol=0.1)


def test_reference_axes_and_bad_positions():
    rng = np.random.default_rng(1)
    cs = rng.standard_normal((9, 2, 8)).astype(np.float32)
    x = rng.standard_normal((1, 2, 1, 16)).astype(np.float32)
    pos = np.array([[[1, 9]], [[4, -1]]])
    got = forms.turned(x, pos, cs, np.array([0, 1, 0, 1, 0, 1, 2, 0]), False)
    assert got[0, 0, 0, 1] == x[0, 0, 0, 1] * cs[4, 0, 1] - x[0, 0, 0, 9] * cs[4, 1, 1]
    assert got[0, 0, 0, 10] == x[0, 0, 0, 10] * cs[1, 0, 2] + x[0, 0, 0, 2] * cs[1, 1, 2]
    assert got[0, 0, 0, 6] == x[0, 0, 0, 6]            # axis 2 of two
    assert np.array_equal(got[0, 1], x[0, 1])          # positions outside the table


def test_reference_visible_positions():
    full = forms.visible(6, 3)
    assert full.sum(1).tolist() == [4, 5, 6]
    assert forms.visible(6, 3, window=2, sinks=1).tolist() == [
        [True, False, True, True, False, False], [True, False, False, True, True, False],
        [True, False, False, False, True, True]]
    # a tree: nodes 1 and 2 are children of the root, 3 of 2
    parent = np.array([-1, 0, 0, 2])
    assert forms.visible(7, 4, parent).tolist() == [
        [True] * 4 + [False] * 3, [True] * 5 + [False] * 2,
        [True] * 4 + [False, True, False], [True] * 4 + [False, True, True]]
    assert forms.visible(7, 4, parent, window=2)[3].tolist() == [False] * 5 + [True, True]
    assert forms.visible(7, 4, parent, window=3, sinks=1)[3].tolist() == \
        [True, False, False, True, False, True, True]
    assert not forms.visible(2, 4, window=1)[:2].any()
    assert forms.visible(2, 4, window=1)[3].tolist() == [False, True]
