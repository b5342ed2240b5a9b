"""The norm and softmax routing without a GPU: pins of the oracle (closed forms, finite differences), and the
host-side refusals of the library's calls (checked before any device call)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU
from workloads import MID, TINY, V3_FP8
from workloads.inputs import rng

BIG = 1 << 40


# ---------------------------------------------------------------- the oracle
def test_norm_closed_form():
    y, r = oracle.rms_norm([[3.0, 4.0], [0.0, 0.0]], [1.0, 2.0], 1e-6)
    assert np.allclose(y[0], np.array([3.0, 8.0]) / np.sqrt(12.5 + 1e-6)) and (y[1] == 0).all() and np.isclose(r[1], 1e3)


def test_norm_backward_by_differences():
    g = rng(91)
    T, H = 3, 7
    h, w, dy, dh = g.standard_normal((T, H)), g.standard_normal(H), g.standard_normal((T, H)), g.standard_normal((T, H))
    f = lambda h, w: (dy * oracle.rms_norm(h, w, 1e-3)[0]).sum() + (dh * h).sum()
    dx, dw = oracle.rms_norm_backward(h, w, 1e-3, dy, dh)
    d = 1e-6
    for i in range(T):
        for j in range(H):
            e = np.zeros((T, H))
            e[i, j] = d
            assert abs((f(h + e, w) - f(h - e, w)) / (2 * d) - dx[i, j]) < 1e-7
    for j in range(H):
        e = np.zeros(H)
        e[j] = d
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * d) - dw[j]) < 1e-7


def test_softmax_affinities():
    x, w = rng(92).standard_normal((5, 8)), rng(93).standard_normal((6, 8))
    s = oracle.affinity_softmax(x, w)
    assert s.dtype == np.float32 and np.allclose(s.sum(axis=1), 1, atol=1e-6)
    o = np.zeros(6)
    o[[1, 4]] = -np.inf
    s = oracle.affinity_softmax(x, w, o)
    assert (s[:, [1, 4]] == 0).all() and np.allclose(s.sum(axis=1), 1, atol=1e-6)
    assert (oracle.affinity_softmax(x, w, np.full(6, -np.inf)) == 0).all()
    assert (oracle.affinity_softmax(x, w, o, ) == s).all()


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("raw", [True, False])
def test_route_backward_by_differences(softmax, raw):
    g = rng(94, softmax, raw)
    T, H, E, k = 4, 5, 6, 2
    x, w, dw = g.standard_normal((T, H)), g.standard_normal((E, H)), g.standard_normal((T, k))

    def s_of(x, w):
        l = x @ w.T
        if not softmax:
            return 1 / (1 + np.exp(-l))
        e = np.exp(l - l.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)

    idx = np.argsort(-s_of(x, w), axis=1)[:, :k]

    def f(x, w):
        s = s_of(x, w)
        sel = np.take_along_axis(s, idx, 1)
        gates = 2.5 * sel if raw else 2.5 * sel / sel.sum(axis=1, keepdims=True)
        return (dw * gates).sum() + oracle.seq_balance_loss(s, idx, k, 2, 0.3)[0]

    dx, dwr, loss = oracle.route_backward(x, w, s_of(x, w), idx, dw, 2.5, 0.3, 2, softmax, raw)
    d = 1e-6
    for a, grad, at in ((x, dx, 0), (w, dwr, 1)):
        for i in np.ndindex(a.shape):
            e = np.zeros(a.shape)
            e[i] = d
            up = f(x + e, w) - f(x - e, w) if at == 0 else f(x, w + e) - f(x, w - e)
            assert abs(up / (2 * d) - grad[i]) < 1e-7


# ---------------------------------------------------------------- refusals: the norm
def test_norm_refusals():
    def norm(c=None, n=None, x=16, res=16, w=16, eps=1e-6, h=16, y=16, q=None, s=None):
        return L.lib().moe_norm(ctypes.byref(c or L.cfg_from(MID)), n, x, res, w, eps, h, y, q, s, None)

    assert norm(x=None) == norm(w=None) == norm(y=None) == L.MOE_ERR_NULL
    c8, ci = L.cfg_from(V3_FP8), L.cfg_from(MID, wgt="int8")
    for c in (c8, ci):
        assert norm(c, q=16) == L.MOE_ERR_NULL                         # codes need a place for their scales
        assert norm(c, q=24, s=16) == norm(c, q=16, s=18) == L.MOE_ERR_UNSUPPORTED
    for c in (L.cfg_from(MID), L.cfg_from(TINY), L.cfg_from(MID, wgt="mxfp4")):
        assert norm(c, q=16, s=16) == L.MOE_ERR_UNSUPPORTED
    for kw in (dict(x=24), dict(res=24), dict(w=24), dict(h=24), dict(y=24), dict(n=18)):
        assert norm(**kw) == L.MOE_ERR_UNSUPPORTED, kw
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(eps=eps) == L.MOE_ERR_SHAPE
    assert norm(L.cfg_from(MID, T=1 << 23, k=1, H=128, I=128)) == L.MOE_ERR_SHAPE
    assert norm(L.cfg_from(MID, T=0), x=None, w=None, y=None) == L.MOE_OK


def test_norm_backward_refusals():
    cfg = L.cfg_from(MID)
    need = L.moe_workspace_bytes(cfg, L.MOE_WS_NORM_BWD)
    assert need >= 512 * MID.H * 4

    def bwd(c=cfg, n=None, h=16, w=16, eps=1e-6, dy=16, dh=16, dx=16, dw=16, ws=16, size=need):
        return L.lib().moe_norm_backward(ctypes.byref(c), n, h, w, eps, dy, dh, dx, dw, ws, size, None)

    assert bwd(h=None) == bwd(w=None) == bwd(dy=None) == bwd(dx=None) == bwd(dw=None) == bwd(ws=None) == L.MOE_ERR_NULL
    for kw in (dict(h=24), dict(w=24), dict(dy=24), dict(dh=24), dict(dx=24), dict(ws=24), dict(dw=18), dict(n=18)):
        assert bwd(**kw) == L.MOE_ERR_UNSUPPORTED, kw
    assert bwd(size=need - 1) == L.MOE_ERR_WORKSPACE
    assert bwd(eps=0.0) == L.MOE_ERR_SHAPE


def test_binding_refusals():
    cfg = L.cfg_from(MID)
    t = torch.zeros((MID.T, MID.H), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.moe_norm(cfg, None, t, None, 16, 1e-6, None, 16, stream=0)
    with pytest.raises(TypeError):
        L.moe_norm(cfg, 7, 16, None, 16, 1e-6, None, 16, stream=0)
    with pytest.raises(ValueError):
        L.moe_norm_backward(cfg, torch.zeros(2, dtype=torch.int32), 16, 16, 1e-6, 16, None, 16, 16, 16, stream=0)


def test_runner_refusals():
    layer = MoeLayerGPU.__new__(MoeLayerGPU)
    layer.c, layer.share, layer.gather, layer.n_tokens, layer.adds_balance = MID, None, False, None, True
    with pytest.raises(ValueError, match="no norm|has none"):
        layer.forward(None, None, residual=object())
    with pytest.raises(ValueError, match="no norm"):
        layer.backward(None, None, dh=object())


def test_runner_refuses_rows_of_another_shape():
    layer = MoeLayerGPU.__new__(MoeLayerGPU)
    layer.c, layer.share, layer.gather, layer.n_tokens, layer.adds_balance = MID, None, False, None, True
    layer.T, layer.act_dtype, layer.norm = 8, torch.bfloat16, object()
    rows = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)
    good = rows(8, MID.H)
    for bad in (rows(7, MID.H), rows(8, MID.H - 8), rows(8 * MID.H), rows(8, MID.H, dtype=torch.float32)):
        with pytest.raises(ValueError, match="residual of shape"):
            layer.forward(good, None, residual=bad)
        with pytest.raises(ValueError, match="x of shape"):
            layer.forward(bad, None, residual=good)
        with pytest.raises(ValueError, match="dh of shape"):
            layer.backward(good, good, dh=bad)


# ---------------------------------------------------------------- refusals: routing flags
def test_route_flags():
    cfg = L.cfg_from(MID)
    f = L.lib().moe_route
    call = lambda flags, scores=16: f(ctypes.byref(cfg), 16, 16, None, 16, scores, flags, None, 16, 16, BIG, None)
    for flags in (0, 1, 2, 4, 5, 6):
        assert call(flags) == L.MOE_ERR_NULL, flags                     # (topk_idx)
    for flags in (3, 7, 8, 10):
        assert call(flags) == L.MOE_ERR_UNSUPPORTED, flags
    assert f(ctypes.byref(cfg), 16, 16, None, 16, None, 2, 16, 16, None, 0, None) == L.MOE_ERR_WORKSPACE


def test_route_backward_flags_refusals():
    cfg = L.cfg_from(MID)
    need = L.moe_workspace_bytes(cfg, L.MOE_WS_ROUTE_BWD_SOFTMAX)
    assert need > L.moe_workspace_bytes(cfg, L.MOE_WS_ROUTE_BWD)

    def bwd(c=cfg, flags=2, x=16, w=16, s=16, idx=16, dw=16, alpha=0.0, seq=0, dx=16, dwr=16, loss=16, ws=16, n=need):
        return L.lib().moe_route_backward_flags(ctypes.byref(c), flags, x, w, s, idx, dw, alpha, seq, dx, dwr, loss, ws, n,
                                                None)

    for flags in (0, 1, 3, 8):
        assert bwd(flags=flags) == L.MOE_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(w=None), dict(s=None), dict(idx=None), dict(dw=None), dict(dwr=None), dict(loss=None),
               dict(ws=None)):
        assert bwd(**kw) == L.MOE_ERR_NULL, kw
    for kw in (dict(x=24), dict(w=24), dict(ws=24), dict(s=18), dict(idx=18), dict(dw=18), dict(dx=18), dict(dwr=18),
               dict(loss=18)):
        assert bwd(**kw) == L.MOE_ERR_UNSUPPORTED, kw
    assert bwd(alpha=-1.0) == bwd(seq=3) == bwd(alpha=float("inf")) == L.MOE_ERR_SHAPE
    assert bwd(n=need - 1) == L.MOE_ERR_WORKSPACE
    assert bwd(c=L.cfg_from(V3_FP8), n=BIG) == bwd(c=L.cfg_from(TINY), n=BIG) == L.MOE_ERR_UNSUPPORTED
