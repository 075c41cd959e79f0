"""CPU checks of the rotary append's rows of q_out: strides that count, and those of an axis of
one, which do not.  (None of these calls reaches the GPU.)"""
import pytest
import torch

import hybrid_gated_deltanet_delta_gb300 as gdn
from test_kv4_forms_host import _tensors


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
