"""Experts out of service: a bias of -inf keeps them out on every selection path, through steps of the bias update; an
offset of -inf alone takes them out of the softmax, not out of the ranking.  Experts bit for bit against the oracle."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU, to_device
from gpu_util import dev_f32, host, say
from workloads import MID
from workloads.inputs import f32_to_bf16_bits, make_weights, make_x, rng

pytestmark = pytest.mark.gpu

# (T, E, G, M, k, topr): a wavefront a token, the fused kernel, 16 lanes a token, the general selection
PATHS = [(9, 256, 8, 4, 8, 2), (2100, 256, 8, 4, 8, 2), (17000, 256, 8, 4, 8, 4), (70, 128, 4, 2, 6, 1),
         (5000, 64, 8, 3, 6, 2), (9, 16, 4, 2, 4, 2), (300, 60, 5, 3, 20, 5), (257, 300, 3, 2, 32, 8), (2100, 160, 8, 3, 6, 2)]


def _inputs(T, E):
    g = rng(221, T, E)
    grid = lambda n, sigma, unit, most: (np.clip(np.rint(g.standard_normal((n, 64)) * sigma / unit), -most, most) * unit
                                         ).astype(np.float32)
    return grid(T, 1.0, 2.0 ** -3, 32), grid(E, 0.2, 2.0 ** -11, 61), g


def _route(cfg, flags, x, w, o, bias, s=None):
    idx = torch.full((cfg.T, cfg.k), -1, dtype=torch.int32, device="cuda")
    gates = torch.full((cfg.T, cfg.k), float("nan"), device="cuda")
    ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_ROUTE), dtype=torch.uint8, device="cuda")
    L.moe_route(cfg, x, w, o, bias, s, flags, idx, gates, ws)
    torch.cuda.synchronize()
    return host(idx), host(gates)


@pytest.mark.parametrize("T,E,G,M,k,topr", PATHS)
def test_masks(T, E, G, M, k, topr):
    say(f"masked experts T={T} E={E} G={G} M={M} k={k}")
    x, w, g = _inputs(T, E)
    xd, wd = (to_device(f32_to_bf16_bits(a)) for a in (x, w))
    cfg = L.make_cfg(T, 64, E, G, M, k, 0, 128, topr, 2.5, "bf16", "bf16")
    out = np.sort(g.permutation(E)[:max(1, E // 8)])
    o = g.standard_normal(E).astype(np.float32)
    o[out] = -np.inf
    s = oracle.affinity_softmax(x, w, o)
    assert (s[:, out] == 0).all()
    bias = (g.uniform(-0.1, 0.1, E) / E).astype(np.float32)
    # a bias above every affinity: the offset alone keeps nobody out of the ranking
    bias[out] = 2
    idx, gates = _route(cfg, L.MOE_SOFTMAX, xd, wd, dev_f32(o), dev_f32(bias))
    ir, gr = oracle.route(s, bias, G, M, k, topr, 2.5)
    assert (idx == ir).all() and np.isin(idx, out).any() and (gates[np.isin(idx, out)] == 0).all()
    # the bias at -inf: out of service, with the offset or without
    bias[out] = -np.inf
    for off, sr in ((o, s), (None, oracle.affinity_softmax(x, w))):
        idx, gates = _route(cfg, L.MOE_SOFTMAX, xd, wd, None if off is None else dev_f32(off), dev_f32(bias))
        ir, gr = oracle.route(sr, bias, G, M, k, topr, 2.5)
        assert (idx == ir).all() and not np.isin(idx, out).any()
        assert (np.abs(gates - gr) <= 40 * 2.0 ** -24 * gr).all()
        idx, _ = _route(cfg, L.MOE_SCORES_IN, None, None, None, dev_f32(bias), dev_f32(sr))
        assert (idx == ir).all()
    # whole groups, and fewer served experts than slots
    bias[E // G:] = -np.inf
    bias[:E // G] = np.where(np.arange(E // G) < (k + 1) // 2, bias[:E // G], -np.inf)
    idx, _ = _route(cfg, L.MOE_SOFTMAX, xd, wd, dev_f32(o), dev_f32(bias))
    ir, _ = oracle.route(s, bias, G, M, k, topr, 2.5)
    assert (idx == ir).all()


@pytest.mark.parametrize("T,E", [(64, 256), (2100, 256), (300, 60)])
def test_a_mask_outlives_the_bias_update(T, E):
    """Steps with a rate that would bring an expert back after two of them."""
    c = MID.with_(T=T, H=128, E=E, G=1, M=1, k=4, S=0, I=128, group_topr=1)
    wts = make_weights(c)
    out = np.array([0, 7, E - 1])
    o = np.zeros(E, np.float32)
    o[out] = -np.inf
    wts.logit_offset = o
    layer = MoeLayerGPU(c, wts, softmax=True)
    bias = wts.bias0.copy()
    bias[out] = -np.inf
    bias = dev_f32(bias)
    say(f"masked experts through updates T={T} E={E}")
    for step in range(5):
        layer.forward(to_device(make_x(c, step)), bias, gamma=0.6)
        torch.cuda.synchronize()
        assert (host(layer.counts)[out] == 0).all() and not np.isin(host(layer.topk_idx), out).any()
        assert (host(bias)[out] == -np.inf).all() and np.isfinite(np.delete(host(bias), out)).all()
        assert np.isfinite(host(layer.y)).all()
