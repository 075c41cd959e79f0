"""CPU checks of the binding's windows and sinks (no call reaches the GPU): any integer counts as
what it is, however large or negative."""
import types

import pytest
import torch

import hybrid_gated_deltanet_delta_gb300 as gdn
from test_kv4_forms_host import _tensors, lib  # noqa: F401

MOST = 2 ** 31 - 1


def bound(monkeypatch, **kw):
    monkeypatch.setattr(gdn, "_on_device", lambda *t: None)
    a = _tensors()
    q = a["q"].to(torch.bfloat16)
    return gdn.bind_kv4_attention_window(q, a["pages"], a["table"], a["kv_len"],
                                         torch.empty_like(q), torch.zeros(16, dtype=torch.uint8),
                                         scale=1.0, stream=types.SimpleNamespace(cuda_stream=0), **kw)


@pytest.mark.parametrize("window, sinks", [(-2 ** 32 + 5, 0), (-2 ** 31, 0), (0, 0), (-1, 3),
                                           (5, -2 ** 32), (5, -2 ** 33 + 7), (5, -1)])
def test_negative_ones_are_refused(monkeypatch, lib, window, sinks):  # noqa: F811
    """The library's numbers are of 32 bits: one past them must not come out as another."""
    with pytest.raises(gdn.GdnError, match="INVALID_ARG"):
        bound(monkeypatch, window=window, sinks=sinks)()


@pytest.mark.parametrize("x", [2 ** 31, 2 ** 32 + 5, 10 ** 30])
def test_large_ones_see_everything(monkeypatch, lib, x):  # noqa: F811
    call = bound(monkeypatch, window=x, sinks=x)
    assert call._args[8:10] == (MOST, MOST)
