"""The balance loss does not depend on which experts a rank holds, so only one share may add it."""
import pytest

from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU
from workloads import MID
from workloads.inputs import make_weights

C = MID.with_(T=8, H=64, E=16, G=4, M=2, k=4, S=1, I=128)


def _record(monkeypatch):
    alphas = []
    for name in ("moe_combine_backward", "moe_combine_local_backward", "moe_expert_ffn_backward",
                 "moe_dispatch_backward", "moe_dispatch_local_backward"):
        monkeypatch.setattr(L, name, lambda *a, **k: None)
    monkeypatch.setattr(L, "moe_route_backward", lambda *a, **k: alphas.append(a[6]))
    return alphas


def test_one_share_adds_the_balance_loss(monkeypatch):
    wts, alphas = make_weights(C), _record(monkeypatch)
    for share in ((0, 7), (7, 9)):
        with pytest.raises(ValueError, match="balance"):
            MoeLayerGPU(C, wts, device="cpu", share=share).backward(None, None, alpha=0.1)
    assert alphas == []
    MoeLayerGPU(C, wts, device="cpu", share=(7, 9)).backward(None, None)
    MoeLayerGPU(C, wts, device="cpu", share=(0, 7), adds_balance=True).backward(None, None, alpha=0.1)
    MoeLayerGPU(C, wts, device="cpu", share=(0, 16)).backward(None, None, alpha=0.2)
    MoeLayerGPU(C, wts, device="cpu").backward(None, None, alpha=0.3)
    assert alphas == [0.0, 0.1, 0.2, 0.3]
