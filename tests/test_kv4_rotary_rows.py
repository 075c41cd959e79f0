"""CPU checks of the rotary append's rows of q_out: strides that count, and those of an axis of
one, which do not.  (None of these calls reaches the GPU.)"""
import pytest
import torch

import hybrid_gated_deltanet_delta_gb300 as gdn
from test_kv4_forms_host import _rotary, _tensors, append_rotary
from test_kv4_host import _cache, lib  # noqa: F401


@pytest.mark.parametrize("B, N, strides", [(1, 3, (64, 256, 64, 1)), (2, 1, (256, 8, 64, 1)),
                                           (1, 1, (24, 40, 64, 1))])
def test_binding_takes_any_stride_of_an_axis_of_one(monkeypatch, B, N, strides):
    """q_out in q's place, whose strides differ on such an axis only: what is refused is that
    these are the host's tensors, the last of the binding's checks."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a = _tensors(B=B, N=N)
    a["q_out"] = a["q"].as_strided(a["q"].shape, strides)
    assert a["q_out"].data_ptr() == a["q"].data_ptr() and a["q_out"].stride() != a["q"].stride()
    with pytest.raises(ValueError, match="current CUDA device"):
        gdn.gdn_kv4_append_rotary(**a)


def test_binding_refuses_other_strides_in_place(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a = _tensors(B=2, N=2)
    a["q_out"] = a["q"].as_strided(a["q"].shape, (256, 512, 64, 1))
    with pytest.raises(ValueError, match="strides"):
        gdn.gdn_kv4_append_rotary(**a)


@pytest.mark.parametrize("B, N, sb, sn", [
    (2, 4, 24576, 0), (2, 4, 0, 6144),        # one row for all nodes, for all sequences
    (2, 4, 24576, 6136), (2, 4, 6136, 24576),  # rows that end in the next
    (2, 4, 18432, 6144),                      # a sequence's last node in the next one's first
    (4, 2, 6144, 18432), (3, 3, 6144, 6144), (2, 4, -6144, 6144),
    (1, 4, 0, 0), (4, 1, 8, 1 << 40),
])
@pytest.mark.parametrize("out", [0x100, 0x200000])   # in place, apart
def test_rows_of_q_out_that_overlap_are_refused(lib, B, N, sb, sn, out):  # noqa: F811
    """24 heads of 256: rows of 6,144 elements.  (Two blocks would write, or in place turn, the
    same queries.)"""
    c, r = _cache(B=B), _rotary()
    assert append_rotary(lib, c, r, q=0x100, qsb=sb, qsn=sn, out=out, osb=sb, osn=sn,
                         N=N) == gdn.GDN_ERR_INVALID_ARG


@pytest.mark.parametrize("Hkv, want", [(65504, gdn.GDN_ERR_UNSUPPORTED), (65536, gdn.GDN_ERR_UNSUPPORTED)])
def test_kv_heads_beside_the_blocks_of_queries(lib, Hkv, want):  # noqa: F811
    """Both stand on one axis of the grid, which has 65,535 places: refused before anything else is
    looked at (the missing queries are a later refusal)."""
    c = _cache(D=64, Hkv=Hkv, page_stride=Hkv * 2 * 36 * 64)
    assert append_rotary(lib, c, _rotary(), q=0, Hq=Hkv, N=1) == want


def test_most_kv_heads(lib):  # noqa: F811
    c = _cache(D=64, Hkv=65503, page_stride=65503 * 2 * 36 * 64)
    assert append_rotary(lib, c, _rotary(), q=0, Hq=65503, N=1) == gdn.GDN_ERR_INVALID_ARG
    # rows of blocks of queries beside them: (blocks of one token) / (records that N tokens touch)
    assert max(-(-N // ((N + 30) // 32 + 1)) for N in range(1, 1 << 16)) <= 32
