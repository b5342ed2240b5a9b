"""Host-side refusals of the share calls (moe_dispatch_local and the calls beside it),
checked before any device call, and of the runner's share and padded batch."""
import ctypes

import pytest
import torch

from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU
from workloads import MID, TINY
from workloads.inputs import make_weights

A = 16   # an aligned address that is never dereferenced


def _cfg(**kw):
    return L.cfg_from(MID, G=1, M=1, **kw)


def test_dispatch_local_refusals():
    cfg = _cfg(E=8)
    need = L.moe_workspace_bytes(cfg, L.MOE_WS_DISPATCH)
    fn = L.lib().moe_dispatch_local
    names = ["first", "n", "idx", "x", "counts", "offsets", "perm", "inv", "x_perm", "scale", "ws", "bytes"]
    base = dict(zip(names, [0, A, A, A, A, A, A, A, A, None, A, need]))

    def call(c=cfg, **kw):
        v = dict(base, **kw)
        return fn(ctypes.byref(c), *(v[n] for n in names), None)

    for n in ("idx", "counts", "offsets", "perm", "inv", "x", "ws"):
        assert call(**{n: None}) == L.MOE_ERR_NULL, n
    assert call(first=-1) == L.MOE_ERR_SHAPE
    assert call(bytes=need - 1) == L.MOE_ERR_WORKSPACE
    for n in ("n", "idx", "counts", "offsets", "perm", "inv", "ws"):
        assert call(**{n: A + 2}) == L.MOE_ERR_UNSUPPORTED, n
    for n in ("x", "x_perm"):
        assert call(**{n: A + 8}) == L.MOE_ERR_UNSUPPORTED, n
    assert call(_cfg(E=5)) == L.MOE_ERR_SHAPE                      # fewer experts than k = 6
    for wgt in ("fp8_e4m3", "mxfp4"):
        assert call(_cfg(E=8, wgt=wgt)) == L.MOE_ERR_NULL          # x_perm needs its scales


def test_combine_local_refusals():
    cfg = _cfg(E=8)
    fn = L.lib().moe_combine_local
    base = [A] * 5
    for i, bad in ((0, None), (1, None), (2, None), (3, None), (4, None)):
        args = list(base)
        args[i] = bad
        assert fn(ctypes.byref(cfg), *args, None) == L.MOE_ERR_NULL, i
        args[i] = A + (8 if i in (0, 1, 4) else 2)
        assert fn(ctypes.byref(cfg), *args, None) == L.MOE_ERR_UNSUPPORTED, i
    assert fn(ctypes.byref(_cfg(E=8, T=0)), *base, None) == L.MOE_OK


def test_backward_local_refusals():
    cfg = _cfg(E=8)
    cb, db = L.lib().moe_combine_local_backward, L.lib().moe_dispatch_local_backward
    for bad in (L.cfg_from(TINY), _cfg(E=8, wgt="fp8_e4m3"), _cfg(E=8, wgt="mxfp4")):
        assert cb(ctypes.byref(bad), *[A] * 6, None) == L.MOE_ERR_UNSUPPORTED
        assert db(ctypes.byref(bad), *[A] * 5, None) == L.MOE_ERR_UNSUPPORTED
    for i in range(6):
        args = [A] * 6
        args[i] = None
        assert cb(ctypes.byref(cfg), *args, None) == L.MOE_ERR_NULL, i
        args[i] = A + (8 if i in (0, 1, 4) else 2)
        assert cb(ctypes.byref(cfg), *args, None) == L.MOE_ERR_UNSUPPORTED, i
    for i in (0, 1, 3, 4):
        args = [A] * 5
        args[i] = None
        assert db(ctypes.byref(cfg), *args, None) == L.MOE_ERR_NULL, i
    for i in range(5):
        args = [A] * 5
        args[i] = A + (2 if i == 3 else 8)
        assert db(ctypes.byref(cfg), *args, None) == L.MOE_ERR_UNSUPPORTED, i
    assert cb(ctypes.byref(_cfg(E=8, T=0)), *[A] * 6, None) == L.MOE_OK
    assert db(ctypes.byref(_cfg(E=8, T=0)), *[A] * 5, None) == L.MOE_OK


def test_batches_past_a_grid_are_refused():
    lib, ws = L.lib(), 1 << 40
    for T, status in ((1 << 23, L.MOE_ERR_SHAPE), ((1 << 23) - 1, L.MOE_ERR_NULL)):
        c = ctypes.byref(_cfg(E=8, T=T))
        assert lib.moe_dispatch_local(c, 0, None, *[A] * 5, None, A, None, A, ws, None) == status
        assert lib.moe_combine_local(c, A, A, A, None, A, None) == status
        assert lib.moe_combine_local_backward(c, A, A, A, None, A, A, None) == status
        assert lib.moe_dispatch_local_backward(c, A, A, None, None, A, None) == status


def test_binding_refuses_strided_tensors():
    cfg = _cfg(E=8, T=4, H=64)
    y = torch.zeros((24, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.moe_combine_local(cfg, y[:, ::2], A, A, A, A, stream=0)


def test_binding_refuses_host_tensors():
    cfg = _cfg(E=8)
    for args in ([torch.zeros(4), A, A, A, A], [A, A, A, A, torch.zeros((2, 2))]):
        with pytest.raises(ValueError):
            L.moe_combine_local(cfg, *args, stream=0)
    L.moe_combine_local(_cfg(E=8, T=0), torch.zeros(0), None, None, None, None, stream=0)


def test_replay_leaves_its_own_batch():
    """A forward pass of a whole batch between a padded graph's replays: backward() after the replay has absent
    pairs again."""
    layer = MoeLayerGPU(TINY, make_weights(TINY), device="cpu")
    n = torch.zeros(1, dtype=torch.int32)
    layer.graph, layer.graph_inputs = type("Graph", (), {"replay": lambda self: None})(), (None, None, n)
    assert not layer.partial
    layer.replay()
    assert layer.partial and layer.n_tokens is n


def test_runner_refuses_bad_shares():
    """Shares outside the layer, smaller than k, or given other experts' weights (before any allocation)."""
    w = make_weights(TINY)
    for share in ((-1, 8), (9, 8), (0, TINY.k - 1), (0, 17)):
        with pytest.raises(ValueError):
            MoeLayerGPU(TINY, w, device="cpu", share=share)
    few = make_weights(TINY.with_(E=5, G=1, M=1))
    with pytest.raises(ValueError):
        MoeLayerGPU(TINY, few, device="cpu", share=(0, 8))


def test_runner_refuses_bias_update_of_a_part():
    layer = MoeLayerGPU(TINY, make_weights(TINY), device="cpu", share=(4, 8))
    assert layer.counts.numel() == 8 and layer.w_gate_up.shape[0] == 8
    with pytest.raises(ValueError):
        layer.forward(None, None, gamma=1e-3)
    with pytest.raises(ValueError):
        layer.update_bias(None, 1e-3)
    whole = MoeLayerGPU(TINY, make_weights(TINY), device="cpu")
    with pytest.raises(ValueError):
        whole.forward(None, None, gamma=1e-3, n_tokens=torch.zeros(1, dtype=torch.int32))
