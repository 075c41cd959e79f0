"""CPU checks of the 4-bit key/value cache: struct layouts, host-side argument
checks of every gdn_kv4_* call (none of these calls reaches the GPU), the
binding's refusals, and the reference's own definitions."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import hybrid_gated_deltanet_delta_gb300 as gdn
import kv4_reference as ref
from hybrid_gated_deltanet_delta_gb300 import build as gdn_build

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load()


@pytest.mark.parametrize("name, struct", [("gdn_kv4_cache", gdn.Kv4Cache),
                                          ("gdn_kv4_pool", gdn.Kv4Pool)])
def test_struct_layout_matches_c(tmp_path, name, struct):
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include "gdn.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void){'
                   f'printf("%zu", sizeof({name}));'
                   + "".join(f'printf(" %zu", offsetof({name}, {f}));' for f in fields)
                   + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", INCLUDE, str(src), "-o", str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    assert got == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


def _cache(**kw):
    c = gdn.Kv4Cache()
    base = dict(pages=0x10000, table=0x20000, kv_len=0x30000, page_stride=4 * 2 * 36 * 256,
                table_stride=8, n_pages=10, page_tokens=64, max_pages=8, B=2, Hkv=4, D=256)
    base.update(kw)
    for key, val in base.items():
        setattr(c, key, val)
    return c


CACHE_CHECKS = [
    (dict(B=-1), gdn.GDN_ERR_INVALID_ARG),
    (dict(Hkv=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(n_pages=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(max_pages=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(D=96), gdn.GDN_ERR_UNSUPPORTED),
    (dict(page_tokens=48), gdn.GDN_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 26, table_stride=1 << 26), gdn.GDN_ERR_UNSUPPORTED),
    (dict(table_stride=7), gdn.GDN_ERR_INVALID_ARG),
    (dict(page_stride=4 * 2 * 36 * 256 - 16), gdn.GDN_ERR_INVALID_ARG),
    (dict(page_stride=4 * 2 * 36 * 256 + 8), gdn.GDN_ERR_MISALIGNED),
    (dict(pages=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(pages=0x10008), gdn.GDN_ERR_MISALIGNED),
    (dict(table=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(kv_len=0x30002), gdn.GDN_ERR_MISALIGNED),
    (dict(k_scale=0x30002), gdn.GDN_ERR_MISALIGNED),
    (dict(status=0x30001), gdn.GDN_ERR_MISALIGNED),
    (dict(B=0, pages=0), gdn.GDN_OK),
]


@pytest.mark.parametrize("change, want", CACHE_CHECKS)
def test_cache_checks(lib, change, want):
    c = ctypes.byref(_cache(**change))
    V = ctypes.c_void_p
    assert lib.gdn_kv4_append(c, V(0x100), V(0x200), gdn.GDN_BF16, 4096, 1024, 4096, 1024, 4,
                              None) == want
    assert lib.gdn_kv4_read(c, V(0x100), V(0x200), gdn.GDN_F32, 4, None) == want
    assert lib.gdn_kv4_attention(c, V(0x100), gdn.GDN_BF16, 4096, 1024, 4, 24, 1.0, None,
                                 V(0x200), None, V(0x300), 1 << 40, None) == want
    assert lib.gdn_kv4_commit(c, 0, 1, 4, None, V(0x100), V(0x200), None) == want


@pytest.mark.parametrize("kw, want", [
    (dict(N=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(dtype=3), gdn.GDN_ERR_INVALID_ARG),
    (dict(k=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(v=0x208), gdn.GDN_ERR_MISALIGNED),
    (dict(sn=1028), gdn.GDN_ERR_MISALIGNED),
    (dict(sb=4100), gdn.GDN_ERR_MISALIGNED),
])
def test_append_checks(lib, kw, want):
    a = dict(N=4, dtype=gdn.GDN_BF16, k=0x100, v=0x200, sb=4096, sn=1024)
    a.update(kw)
    V = ctypes.c_void_p
    c = ctypes.byref(_cache())
    assert lib.gdn_kv4_append(c, V(a["k"]), V(a["v"]), a["dtype"], a["sb"], a["sn"], a["sb"],
                              a["sn"], a["N"], None) == want
    if "sn" not in kw and "sb" not in kw:
        assert lib.gdn_kv4_read(c, V(a["k"]), V(a["v"]), a["dtype"], a["N"], None) == want


@pytest.mark.parametrize("kw, want", [
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
])
def test_attention_checks(lib, kw, want):
    a = dict(N=4, Hq=24, dtype=gdn.GDN_BF16, q=0x100, o=0x200, sb=4096, sn=1024, parent=0, lse=0,
             ws=0x300, bytes=1 << 40)
    a.update(kw)
    V = ctypes.c_void_p
    assert lib.gdn_kv4_attention(ctypes.byref(_cache()), V(a["q"]), a["dtype"], a["sb"], a["sn"],
                                 a["N"], a["Hq"], 1.0, V(a["parent"]), V(a["o"]), V(a["lse"]),
                                 V(a["ws"]), a["bytes"], None) == want


def test_workspace_sizes(lib):
    assert lib.gdn_kv4_attention_workspace_bytes(8, 16, 24, 4, 256) > 0
    assert lib.gdn_kv4_attention_workspace_bytes(0, 16, 24, 4, 256) == 0
    assert lib.gdn_kv4_attention_workspace_bytes(8, 16, 25, 4, 256) == 0
    assert lib.gdn_kv4_attention_workspace_bytes(8, 16, 24, 4, 80) == 0
    assert lib.gdn_kv4_reserve_workspace_bytes(5) > 0
    assert lib.gdn_kv4_reserve_workspace_bytes(0) == 0


@pytest.mark.parametrize("kw, want", [
    (dict(layers=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(layers=2, stride=16), gdn.GDN_ERR_INVALID_ARG),
    (dict(stride=8), gdn.GDN_ERR_MISALIGNED),
    (dict(N=65, parent=0x400), gdn.GDN_ERR_UNSUPPORTED),
    (dict(accept=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(out=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(out=0x30000), gdn.GDN_ERR_INVALID_ARG),   # kv_len itself
    (dict(accept=0x102), gdn.GDN_ERR_MISALIGNED),
])
def test_commit_checks(lib, kw, want):
    a = dict(layers=1, stride=0, N=4, parent=0, accept=0x100, out=0x200)
    a.update(kw)
    V = ctypes.c_void_p
    assert lib.gdn_kv4_commit(ctypes.byref(_cache()), a["stride"], a["layers"], a["N"],
                              V(a["parent"]), V(a["accept"]), V(a["out"]), None) == want


def _pool(**kw):
    p = gdn.Kv4Pool()
    base = dict(table=0x10000, kv_len=0x20000, ref=0x30000, table_stride=8, n_rows=4, max_pages=8,
                n_pages=100, page_tokens=64)
    base.update(kw)
    for key, val in base.items():
        setattr(p, key, val)
    return p


@pytest.mark.parametrize("change, F, want", [
    (dict(n_rows=0), 1, gdn.GDN_ERR_INVALID_ARG),
    (dict(n_pages=0), 1, gdn.GDN_ERR_INVALID_ARG),
    (dict(page_tokens=40), 1, gdn.GDN_ERR_UNSUPPORTED),
    (dict(table_stride=4), 1, gdn.GDN_ERR_INVALID_ARG),
    (dict(ref=0), 1, gdn.GDN_ERR_INVALID_ARG),
    (dict(ref=0x30002), 1, gdn.GDN_ERR_MISALIGNED),
    (dict(), -1, gdn.GDN_ERR_INVALID_ARG),
    (dict(), 1 << 17, gdn.GDN_ERR_UNSUPPORTED),
    (dict(), 0, gdn.GDN_OK),
])
def test_pool_checks(lib, change, F, want):
    p, V = ctypes.byref(_pool(**change)), ctypes.c_void_p
    assert lib.gdn_kv4_release(p, V(0x100), V(0x200), F, None) == want
    assert lib.gdn_kv4_fork(p, V(0x100), V(0x200), F, None) == want
    assert lib.gdn_kv4_reserve(p, V(0x1000), 4 * 2 * 36 * 256, 1 << 40, 2, 4, 256, V(0x100),
                               V(0x200), F, V(0x3000), 1 << 30, None) == want


@pytest.mark.parametrize("kw, want", [
    (dict(layers=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(D=32), gdn.GDN_ERR_UNSUPPORTED),
    (dict(ps=16), gdn.GDN_ERR_INVALID_ARG),
    (dict(ls=16), gdn.GDN_ERR_INVALID_ARG),
    (dict(pages=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(pages=0x1008), gdn.GDN_ERR_MISALIGNED),
    (dict(ws=0), gdn.GDN_ERR_WORKSPACE),
    (dict(wb=8), gdn.GDN_ERR_WORKSPACE),
])
def test_reserve_checks(lib, kw, want):
    a = dict(pages=0x1000, ps=4 * 2 * 36 * 256, ls=1 << 40, layers=2, D=256, ws=0x3000, wb=1 << 20)
    a.update(kw)
    V = ctypes.c_void_p
    assert lib.gdn_kv4_reserve(ctypes.byref(_pool()), V(a["pages"]), a["ps"], a["ls"],
                               a["layers"], 4, a["D"], V(0x100), V(0x200), 2, V(a["ws"]), a["wb"],
                               None) == want


def test_binding_refuses_bad_tensors(lib):
    i32 = torch.int32
    pages = torch.zeros(4, 2, 2, 36 * 64, dtype=torch.uint8)
    table, kv_len = torch.zeros(1, 2, dtype=i32), torch.zeros(1, dtype=i32)
    k = torch.zeros(1, 3, 2, 64)
    for bad in (dict(pages=pages.float()), dict(pages=pages[..., :100]), dict(pages=pages[0]),
                dict(table=table.long()), dict(kv_len=kv_len.long()),
                dict(table=torch.zeros(2, 2, dtype=i32)), dict(k=k.transpose(1, 2)),
                dict(v=k.half()), dict(k=torch.zeros(1, 3, 2, 32)),
                dict(k_scale=torch.ones(3))):
        a = dict(k=k, v=k, pages=pages, table=table, kv_len=kv_len, k_scale=None)
        a.update(bad)
        with pytest.raises(ValueError):
            gdn.gdn_kv4_append(a["k"], a["v"], a["pages"], a["table"], a["kv_len"],
                               k_scale=a["k_scale"])
    q = torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    for bad in (dict(o=q.float()), dict(o=q[:, :2]), dict(parent=torch.zeros(1, 2, dtype=i32)),
                dict(lse=torch.zeros(1, 3, 4, dtype=torch.float64))):
        a = dict(o=q.clone(), parent=None, lse=None)
        a.update(bad)
        with pytest.raises(ValueError):
            gdn.gdn_kv4_attention(q, pages, table, kv_len, a["o"], ws, scale=1.0,
                                  parent=a["parent"], lse=a["lse"])
    with pytest.raises(ValueError):
        gdn.gdn_kv4_reserve(pages, table, kv_len, torch.zeros(3, dtype=i32), kv_len, kv_len, ws)
    with pytest.raises(TypeError):
        gdn.gdn_kv4_append(k.double(), k.double(), pages, table, kv_len)


# ---- the reference itself
def test_reference_scale_grid_matches_a_cast():
    x = torch.linspace(0, 448, 20001)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref._nearest(ref.E4M3, x.numpy()), want)


def test_reference_codes_are_nearest_values():
    """Every code's value is within half a step of the scaled input, ties to even."""
    x = np.array([[[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5,
                    -3.5, -5.0, -6.0]]])
    code, s8 = ref.quantise(x, np.ones(1))
    assert ref.E4M3[s8[0, 0, 0]] == 1.0
    want = [0, 1, 1, 2, 2, 4, 4, 6, -0.0, -1, -1, -2, -2, -4, -4, -6]
    assert np.array_equal(ref.values(code, s8)[0, 0], want)


def test_reference_put_and_get_are_inverse():
    rng = np.random.default_rng(0)
    D = 64
    cache = ref.Cache(rng.integers(0, 256, (2, 2, 2, 36 * D), dtype=np.uint8), D)
    tok = [rng.integers(0, 16, D).astype(np.uint8), rng.integers(0, 127, D // 16).astype(np.uint8),
           rng.integers(0, 16, D).astype(np.uint8), rng.integers(0, 127, D // 16).astype(np.uint8)]
    others = [cache.get(1, 1, s) for s in (36, 38, 5)]
    others = [[x.copy() for x in t] for t in others]
    cache.put(1, 1, 37, *tok)
    for got, want in zip(cache.get(1, 1, 37), tok):
        assert np.array_equal(got, want)
    for s, want in zip((36, 38, 5), others):
        for got, w in zip(cache.get(1, 1, s), want):
            assert np.array_equal(got, w)


def test_reference_attention_agrees_with_differences_of_lse():
    """The gradient of lse(q) is scale * sum p k: central differences of the reference."""
    rng = np.random.default_rng(1)
    D, P = 64, 32
    cache = ref.Cache(np.zeros((2, 1, 1, 36 * D), np.uint8), D)
    table, kv_len = np.array([[1, 0]]), np.array([40])
    ones = np.ones(1)
    ref.append(cache, table, kv_len, P, rng.standard_normal((1, 40, 1, D)),
               rng.standard_normal((1, 40, 1, D)), ones, ones)
    q, d = rng.standard_normal((1, 1, 1, D)), rng.standard_normal(D)
    lse = [ref.attention(cache, table, kv_len, P, q + e * d, 0.2, ones, ones)[1][0, 0, 0]
           for e in (-1e-4, 1e-4, 0)]
    k, _ = ref.sequence(cache, table[0], 40, P, 0, ones, ones)
    p = np.exp(0.2 * k @ q[0, 0, 0] - lse[2])
    assert abs(p.sum() - 1) < 1e-12
    assert abs((lse[1] - lse[0]) / 2e-4 - 0.2 * p @ k @ d) < 1e-6
