"""Rows that the runner hands to the norm's gradients are checked as forward() checks them."""
import pytest
import torch

from biased_top_routing_amd.runner import MoeLayerGPU
from workloads import MID


def _layer(gather):
    layer = MoeLayerGPU.__new__(MoeLayerGPU)
    layer.c, layer.share, layer.gather, layer.n_tokens, layer.adds_balance = MID, None, gather, None, True
    layer.T, layer.act_dtype, layer.norm = 8, torch.bfloat16, object()
    return layer


def test_backward_refuses_an_x_that_the_norm_would_read_past():
    layer = _layer(False)
    rows = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)
    good = rows(8, MID.H)
    for bad in (rows(7, MID.H), rows(8, MID.H - 8), rows(8 * MID.H), rows(8, MID.H, dtype=torch.float32)):
        with pytest.raises(ValueError, match="x of shape"):
            layer.backward(bad, good)


def test_backward_after_a_residual_does_not_read_x():
    layer = _layer(True)
    layer.residual = object()
    with pytest.raises(ValueError, match="gather=False"):      # (the next refusal)
        layer.backward(None, None)


def test_backward_refuses_affinities_that_were_not_kept(monkeypatch):
    """Without keep_scores the forward pass leaves .scores unwritten, unless the affinities were given."""
    from biased_top_routing_amd import _lib as L
    layer = _layer(False)
    layer.norm, layer.keep_scores, layer.alloc_backward = None, False, lambda: (_ for _ in ()).throw(KeyError("allocates"))
    layer.cfg = layer.w_router = layer.logit_offset = layer.scores = layer.topk_idx = layer.topk_w = layer.ws_route = None
    monkeypatch.setattr(L, "moe_route", lambda *a: None)
    layer.route(None, None)
    with pytest.raises(ValueError, match="keep_scores"):
        layer.backward(None, None)
    layer.route(None, None, scores_in=True)
    with pytest.raises(KeyError):                              # (past the refusals)
        layer.backward(None, None)
    layer.graph_inputs, layer.graph, layer.y = (None, None, None), type("G", (), {"replay": lambda self: None})(), None
    layer.replay()
    with pytest.raises(ValueError, match="keep_scores"):
        layer.backward(None, None)
