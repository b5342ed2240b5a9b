"""MXFP4 expert GEMMs whose workgroups take several tiles of 256 or 288 rows, one after the other: the loads run on into
the next tile while the last one is multiplied, so its descriptors, its rows' entries of perm and the stage in which the
last tile's results are staged all change hands.  Rows sorted, and gathered through perm; odd and even numbers of K
steps, one step; one to three shared experts; segments of one and two tiles, one of them nearly empty, one empty."""
import numpy as np
import pytest
import torch

from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU, to_device
from gpu_util import dev_f32, host, say
from test_gpu_mxfp4 import _check_h, _check_y, _part, _spread, _values
from workloads import MID
from workloads.inputs import make_weights, make_x, rng
import oracle.mxfp4 as mx

pytestmark = pytest.mark.gpu

CASES = [
    # (rows a tile, GEMM whose workgroups take several, T, H, E, k, S, I)
    (256, "gate/up", 130, 128, 6, 6, 1, 11008),
    (256, "gate/up", 130, 384, 6, 6, 1, 5120),
    (256, "gate/up", 250, 256, 5, 5, 2, 5120),
    (256, "down", 130, 10240, 6, 6, 1, 384),
    (256, "down", 200, 9344, 7, 7, 3, 128),
    (288, "gate/up", 260, 128, 6, 6, 1, 7168),
    (288, "gate/up", 270, 384, 6, 6, 1, 5120),
    (288, "gate/up", 280, 256, 5, 5, 2, 5120),
    (288, "gate/up", 550, 384, 4, 2, 1, 5120),
    (288, "down", 260, 10240, 6, 6, 1, 384),
    (288, "down", 550, 10240, 4, 2, 3, 128),
]


def _affinities(T, E, k):
    """Affinities that send every token to all k = E experts, or tokens of T = 550 to experts of 550, 250, 300 and 0."""
    s = np.full((T, E), 0.5, np.float32)
    if k < E:
        t = np.arange(T)
        s[:] = 0.1
        s[t, 0] = 0.9
        s[t, np.where(t % 11 < 5, 1, 2)] = 0.6
    return s


@pytest.mark.parametrize("rows,gemm,T,H,E,k,S,I", CASES)
def test_several_tiles_a_workgroup(rows, gemm, T, H, E, k, S, I):
    say(f"{rows}-row tiles, several a workgroup in {gemm}: T={T} H={H} E={E} k={k} S={S} I={I}")
    c = MID.with_(T=T, H=H, E=E, G=1, M=1, k=k, S=S, I=I, sigma=0.05, group_topr=1, wgt="mxfp4")
    wts, g = make_weights(c), rng(65, T, H, I)
    for name in ("w_gate_up", "w_down", "ws_gate_up", "ws_down"):
        setattr(wts, name, _spread(getattr(wts, name), g))
    xb = _spread(make_x(c), g)
    x, bias = to_device(xb), dev_f32(np.zeros(E))
    layer = MoeLayerGPU(c, wts)
    layer.scores.copy_(dev_f32(_affinities(T, E, k)))
    layer.y_perm.fill_(float("nan"))
    layer.forward(x, bias, scores_in=True)
    torch.cuda.synchronize()
    hdr = host(layer.ws_ffn[:64].view(torch.int32))      # tiles of either GEMM, and the height that was chosen
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert hdr[6] == rows and hdr[0 if gemm == "gate/up" else 1] > cus, hdr[:8]
    offsets, tok = host(layer.offsets), host(layer.perm) // k
    if k < E:
        assert np.diff(offsets).tolist() == [550, 250, 300, 0]
    want = layer.y_perm.clone(), layer.y_shared.clone()

    say("  rows gathered, phases apart")
    for phases, gather in (((L.MOE_FFN_ALL,), True), ((L.MOE_FFN_GATE_UP, L.MOE_FFN_DOWN), True),
                           ((L.MOE_FFN_ALL,), False)):
        layer.y_perm.fill_(float("nan"))
        layer.y_shared.fill_(float("nan"))
        layer.ws_ffn.fill_(0xFF)
        for ph in phases:
            if gather:
                L.moe_expert_ffn_gather(layer.cfg, x, layer.perm, layer.offsets, layer.weights, layer.y_perm,
                                        layer.y_shared, layer.ws_ffn, ph)
            else:
                layer.expert_ffn(x, ph)
        torch.cuda.synchronize()
        for got, ref in zip((layer.y_perm, layer.y_shared), want):
            assert torch.equal(got.view(torch.int16), ref.view(torch.int16)), (phases, gather)

    say("  h and y against 64 bits")                     # a third of the rows of every tile, and its last ones
    xq = _values(xb)
    hq, he = _part(layer, L.MOE_WSP_H, T * k, I)
    yp = host(layer.y_perm)
    pick = lambda n, i: np.flatnonzero((np.arange(n) % 3 == i % 3) | (np.arange(n) % rows >= rows - 3) |
                                       (np.arange(n) >= n - 5))
    for e in range(E):
        r = int(offsets[e]) + pick(int(offsets[e + 1] - offsets[e]), e)
        if r.size:
            _check_h(xq[tok[r]], _values(wts.w_gate_up[e]), hq[r], he[r])
            _check_y(yp[r], [(mx.dequantize_mxfp4(hq[r], he[r]), _values(wts.w_down[e]))])
    hq, he = _part(layer, L.MOE_WSP_H_SHARED, T, S * I)
    r, parts = pick(T, 1), []
    for s in range(S):
        cs, es = slice(s * I, (s + 1) * I), slice(s * I // 32, (s + 1) * I // 32)
        _check_h(xq[r], _values(wts.ws_gate_up[s]), hq[r, cs], he[r, es])
        parts.append((mx.dequantize_mxfp4(hq[r, cs], he[r, es]), _values(wts.ws_down[s])))
    _check_y(host(layer.y_shared)[r], parts)
