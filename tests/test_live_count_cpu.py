"""The live count of a padded batch (n_tokens) is read on the device: whatever is no int32 tensor of one element
there is refused before anything is launched."""
import pytest
import torch

from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU
from workloads import MID, TINY
from workloads.inputs import make_weights

A = 16   # an aligned address that is never dereferenced
I32 = dict(dtype=torch.int32)
BAD = {
    "a number": (TypeError, 96),                       # would be read as an address
    "zero": (TypeError, 0),                            # would be read as "every token"
    "a truth value": (TypeError, True),
    "a list": (TypeError, [96]),
    "64 bits": (ValueError, torch.tensor([96])),
    "float": (ValueError, torch.tensor([96.0])),
    "two": (ValueError, torch.zeros(2, **I32)),
    "none": (ValueError, torch.zeros(0, **I32)),       # no address: would be read as "every token"
    "on the host": (ValueError, torch.tensor([96], **I32)),
}


def _no_launch(monkeypatch):
    for name in ("moe_route", "moe_dispatch", "moe_dispatch_local"):
        monkeypatch.setattr(L, name, lambda *a, **k: pytest.fail("launched"))


@pytest.mark.parametrize("name", BAD)
@pytest.mark.parametrize("share", [None, (4, 8)])
def test_runner_refuses_live_counts(monkeypatch, name, share):
    kind, n = BAD[name]
    layer = MoeLayerGPU(TINY, make_weights(TINY), device="cpu", share=share)
    _no_launch(monkeypatch)
    with pytest.raises(kind, match="n_tokens|no GPU can read"):
        layer.forward(None, None, n_tokens=n)
    assert layer.n_tokens is None
    with pytest.raises(kind, match="n_tokens|no GPU can read"):
        layer.capture(None, None, n_tokens=n)


@pytest.mark.parametrize("name", BAD)
def test_binding_refuses_live_counts(monkeypatch, name):
    kind, n = BAD[name]

    cfg = L.cfg_from(MID, E=8, G=1, M=1)

    class Library:
        def moe_dispatch_local(self, *args):
            pytest.fail("called")

    monkeypatch.setattr(L, "lib", Library)
    with pytest.raises(kind, match="n_tokens|no GPU can read"):
        L.moe_dispatch_local(cfg, 0, n, *[A] * 8, None, stream=0)
