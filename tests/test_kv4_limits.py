"""Sizes of the gdn_kv4_* calls at which a count would pass 32 bits: refused on the host
before anything is launched, and answered by the size functions without a fault."""
import ctypes

import pytest
import torch

import hybrid_gated_deltanet_delta_gb300 as gdn
from hybrid_gated_deltanet_delta_gb300 import build as gdn_build

V = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load()


def reserve(lib, *, F=2, Hkv=4, D=256, page_tokens=64, page_stride=None, **kw):
    p = gdn.Kv4Pool()
    base = dict(table=0x10000, kv_len=0x20000, ref=0x30000, table_stride=8, n_rows=4, max_pages=8,
                n_pages=100, page_tokens=page_tokens)
    base.update(kw)
    for key, val in base.items():
        setattr(p, key, val)
    stride = page_stride or Hkv * (page_tokens // 32) * 36 * D
    return lib.gdn_kv4_reserve(ctypes.byref(p), V(0x1000), stride, 0, 1, Hkv, D, V(0x100),
                               V(0x200), F, V(0x3000), 1 << 40, None)


@pytest.mark.parametrize("F, max_pages", [(65535, 32769), (60000, 60_000_000), (50, 60_000_000)])
def test_reserve_refuses_more_pages_than_it_can_count(lib, F, max_pages):
    assert F * max_pages > 0x7fffffff
    assert reserve(lib, F=F, n_rows=65535, max_pages=max_pages, table_stride=max_pages,
                   page_tokens=32) == gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("records", [3728264, 3728269])
def test_reserve_refuses_pages_that_its_copy_cannot_index(lib, records):
    """Pages of almost 2^31 units of 16 bytes: the copy's next index would pass 32 bits."""
    assert 0x7fffffff - 4095 < records * 36 * 256 // 16 <= 0x7fffffff
    assert reserve(lib, Hkv=1, page_tokens=32 * records, max_pages=1,
                   table_stride=1) == gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("n_pages", [0x7fffffff, 0x7fffffff - 4094])
def test_reserve_refuses_more_counts_than_its_plan_can_index(lib, n_pages):
    assert reserve(lib, n_pages=n_pages) == gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("N, Hq", [(1 << 29, 8), (1 << 24, 4096), (1 << 24, 256), (1 << 23, 256),
                                   (400_000_000, 6), ((1 << 24) + 1, 1), (1 << 24, 65)])
def test_attention_workspace_of_sizes_that_are_refused_is_0(lib, N, Hq):
    """As for the other sizes that gdn_kv4_attention refuses; rows past 2^31 divided by 0."""
    assert lib.gdn_kv4_attention_workspace_bytes(1, N, Hq, 1, 256) == 0


def test_attention_workspace_of_the_largest_call(lib):
    assert lib.gdn_kv4_attention_workspace_bytes(1, 1 << 24, 64, 1, 256) > 0


def test_reserve_granted_checks(lib):
    p = gdn.Kv4Pool()
    for key, val in dict(table=0x10000, kv_len=0x20000, ref=0x30000, table_stride=8, n_rows=4,
                         max_pages=8, n_pages=100, page_tokens=64).items():
        setattr(p, key, val)
    for granted, F, want in ((0, 2, gdn.GDN_ERR_INVALID_ARG), (0x502, 2, gdn.GDN_ERR_MISALIGNED),
                             (0, 0, gdn.GDN_OK), (0x500, -1, gdn.GDN_ERR_INVALID_ARG),
                             (0x500, 1 << 17, gdn.GDN_ERR_UNSUPPORTED)):
        assert lib.gdn_kv4_reserve_granted(ctypes.byref(p), V(0x1000), 4 * 2 * 36 * 256, 0, 1, 4,
                                           256, V(0x100), V(0x200), F, V(granted), V(0x3000),
                                           1 << 20, None) == want


def test_binding_refuses_a_bad_granted(lib):
    i32 = torch.int32
    pages = torch.zeros(4, 2, 2, 36 * 64, dtype=torch.uint8)
    table, one = torch.zeros(1, 2, dtype=i32), torch.zeros(1, dtype=i32)
    for bad in (torch.zeros(2, dtype=i32), torch.zeros(1), torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(ValueError):
            gdn.gdn_kv4_reserve(pages, table, one, torch.zeros(4, dtype=i32), one, one, pages,
                                granted=bad)
