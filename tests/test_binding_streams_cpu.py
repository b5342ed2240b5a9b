"""The binding asks torch for the current device and stream, by torch's internal queries where it has them."""
import types

import pytest
import torch

from biased_top_routing_amd import _lib as L


@pytest.mark.parametrize("internal", [True, False])
def test_current_stream_without_internal_names(monkeypatch, internal):
    monkeypatch.setattr(L, "_device_fn", None)
    monkeypatch.setattr(L, "_stream_fn", None)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    names = dict(_cuda_getDevice=lambda: 3, _cuda_getCurrentRawStream=lambda device: 100 + device)
    monkeypatch.setattr(torch, "_C", types.SimpleNamespace(**(names if internal else {})))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 5)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=200 + d))
    want = 103 if internal else 205
    assert L._s(None) == want and L._s(None) == want       # the first call and later ones
    assert L._device() == (3 if internal else 5)
