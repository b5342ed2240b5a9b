"""int8 without a GPU: pins of the oracle's rule, and the host-side refusals of the library's int8 calls (checked
before any device call)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from oracle.int8 import round_bf16
from workloads import MID, V3_FP8
from workloads.inputs import f32_to_bf16_bits, rng

BIG = 1 << 40


# ---------------------------------------------------------------- the oracle's rule
def test_codes_by_hand():
    q, s = oracle.quantize_int8([[1.0, -2.0, 0.5, 127.0], [254.0, 1.0, 3.0, -5.0], [0, 0, 0, 0]])
    assert q.tolist() == [[1, -2, 0, 127], [127, 0, 2, -2], [0, 0, 0, 0]]      # 0.5, 1.5, -2.5: ties to even
    assert s.tolist() == [1.0, 2.0, 0.0]


def test_no_value_is_off_by_more_than_half_a_step():
    v = rng(81, 1).standard_normal((64, 384)) * np.exp2(rng(81, 2).integers(-30, 30, (64, 1)))
    q, s = oracle.quantize_int8(v)
    assert np.abs(q).max(axis=1).tolist() == [127] * 64
    assert (np.abs(q * s[:, None] - v) <= s[:, None] * (0.5 + 1e-12)).all()


def test_special_rows():
    v = np.ones((3, 8))
    v[0, 3], v[1, 5] = np.nan, -np.inf
    q, s = oracle.quantize_int8(v)
    assert np.isnan(s[:2]).all() and (q[:2] == 0).all() and s[2] == 1 / 127


def test_quotients_of_bf16_values_keep_clear_of_halves():
    """What makes the codes independent of who computes them: in fp32 127 v is exact and 127 v / a, rounded once,
    is a half only where the quotient itself is one (every bf16 significand against every other, a few binades)."""
    a = np.arange(128, 256, dtype=np.float32)
    v = np.arange(128, 256, dtype=np.float32)
    for shift in range(0, 9):
        n = np.float32(127) * (v * np.float32(2.0 ** -shift))
        q32 = n[:, None] / a[None, :]
        assert q32.dtype == np.float32
        exact2 = 2 * 127 * v.astype(np.int64)[:, None]                         # 2 * 127 v over a * 2^shift
        half = (exact2 % (a.astype(np.int64)[None, :] << shift) == 0) & ((exact2 // (a.astype(np.int64) << shift)) % 2 == 1)
        assert ((q32 % 1 == 0.5) == half).all()


def test_round_bf16_is_the_conversion():
    v = rng(82).standard_normal(4096).astype(np.float32)
    assert (round_bf16(v) == oracle.decode_act(f32_to_bf16_bits(v))).all()


# ---------------------------------------------------------------- refusals
def _cfg(**kw):
    return L.cfg_from(MID, **{"wgt": "int8", **kw})


@pytest.mark.parametrize("kw,ok", [
    ({}, True), (dict(act="f32"), False), (dict(H=2048 + 64), False), (dict(I=1408 + 64), False),
    (dict(S=0, E=8, G=1, M=1, k=1, I=128, H=(1 << 17) - 128), True), (dict(S=0, E=8, G=1, M=1, k=1, I=128, H=1 << 17), False),
    (dict(S=93, I=1408, H=128), True), (dict(S=94, I=1408, H=128), False),
    (dict(T=(1 << 26) // 7, H=128, I=128), True), (dict(T=(1 << 26) // 7 + 1, H=128, I=128), False),
])
def test_configurations(kw, ok):
    assert (L.moe_workspace_bytes(_cfg(**kw), L.MOE_WS_FFN) > 0) == ok


def test_workspace_parts():
    cfg = _cfg()
    total = L.moe_workspace_bytes(cfg, L.MOE_WS_FFN)
    P, T, SI = MID.T * MID.k, MID.T, MID.S * MID.I
    want = [P * MID.I, P * 4, T * SI, T * 4]
    end = 0
    for part, n in zip((L.MOE_WSP_H, L.MOE_WSP_H_SCALE, L.MOE_WSP_H_SHARED, L.MOE_WSP_H_SHARED_SCALE), want):
        off, size = L.moe_ffn_workspace_part(cfg, part)
        assert off >= end and n <= size < n + 256 and off % 256 == 0
        end = off + size
    assert end <= total


def test_quantize_refusals():
    f = L.lib().moe_quantize_int8
    assert f(16, 2, 4, 12, 1, 16, 16, None) == L.MOE_ERR_SHAPE          # cols % 8
    assert f(16, 3, 4, 16, 2, 16, 16, None) == L.MOE_ERR_SHAPE          # n_mat % group
    assert f(16, 3, 4, 16, 0, 16, 16, None) == L.MOE_ERR_SHAPE
    assert f(16, -1, 4, 16, 1, 16, 16, None) == L.MOE_ERR_SHAPE
    assert f(16, 1 << 13, 1 << 13, 16, 1, 16, 16, None) == L.MOE_ERR_SHAPE
    assert f(None, 1, 4, 16, 1, 16, 16, None) == L.MOE_ERR_NULL
    assert f(16, 1, 4, 16, 1, None, 16, None) == L.MOE_ERR_NULL
    assert f(16, 1, 4, 16, 1, 16, None, None) == L.MOE_ERR_NULL
    assert f(8, 1, 4, 16, 1, 16, 16, None) == L.MOE_ERR_UNSUPPORTED
    assert f(16, 1, 4, 16, 1, 20, 16, None) == L.MOE_ERR_UNSUPPORTED
    assert f(16, 1, 4, 16, 1, 16, 18, None) == L.MOE_ERR_UNSUPPORTED
    assert f(None, 0, 4, 16, 1, None, None, None) == L.MOE_OK


def _weights(cfg, **kw):
    d = dict(w_gate_up=16, w_down=16, w_gate_up_scale=16, w_down_scale=16, ws_gate_up=16, ws_down=16,
             ws_gate_up_scale=16, ws_down_scale=16)
    d.update(kw)
    return L.MoeExpertWeights(**d)


def test_ffn_refusals():
    cfg = _cfg()
    need = L.moe_workspace_bytes(cfg, L.MOE_WS_FFN)
    r = ctypes.byref(cfg)

    def codes(xc=16, xs=16, perm=16, off=16, w=None, y=16, ys=16, ws=16, n=need, phase=0, c=r):
        return L.lib().moe_expert_ffn_codes(c, xc, xs, perm, off, ctypes.byref(w or _weights(cfg)), y, ys, ws, n, phase,
                                            None)

    assert codes(xc=None) == codes(xs=None) == codes(perm=None) == codes(off=None) == codes(y=None) == codes(ws=None) \
        == codes(ys=None) == L.MOE_ERR_NULL
    for name in ("w_gate_up", "w_down", "w_gate_up_scale", "w_down_scale", "ws_gate_up", "ws_down", "ws_gate_up_scale",
                 "ws_down_scale"):
        assert codes(w=_weights(cfg, **{name: None})) == L.MOE_ERR_NULL, name
        assert codes(w=_weights(cfg, **{name: 18})) == L.MOE_ERR_UNSUPPORTED, name
    assert codes(xc=24) == codes(xs=18) == codes(y=24) == codes(ys=24) == codes(ws=24) == L.MOE_ERR_UNSUPPORTED
    assert codes(n=need - 1) == L.MOE_ERR_WORKSPACE
    assert codes(phase=3) == L.MOE_ERR_UNSUPPORTED
    for other in ("bf16", "mxfp4"):
        assert codes(c=ctypes.byref(_cfg(wgt=other))) == L.MOE_ERR_UNSUPPORTED
    # the FP8 experts take codes too, and check them likewise
    c8 = L.cfg_from(V3_FP8)
    assert codes(c=ctypes.byref(c8), xs=None) == L.MOE_ERR_NULL
    assert codes(c=ctypes.byref(c8), xc=24) == L.MOE_ERR_UNSUPPORTED
    # rows gathered by 32-bit offsets
    big = L.cfg_from(MID, wgt="int8", T=(1 << 20), k=6, H=2048)
    assert codes(c=ctypes.byref(big), n=BIG) == L.MOE_ERR_UNSUPPORTED
    # the sorted rows need their scales
    f = L.lib().moe_expert_ffn
    assert f(r, 16, None, 16, ctypes.byref(_weights(cfg)), 16, 16, 16, 16, need, 0, None) == L.MOE_ERR_NULL
    assert L.lib().moe_dispatch(r, 16, 16, 16, 16, 16, 16, 16, None, 16, BIG, None) == L.MOE_ERR_NULL
    assert L.lib().moe_dispatch(r, 16, 16, 16, 16, 16, 16, 24, 16, 16, BIG, None) == L.MOE_ERR_UNSUPPORTED


def test_training_is_refused():
    cfg = ctypes.byref(_cfg())
    assert L.lib().moe_combine_backward(cfg, 16, 16, 16, 16, 16, 16, None) == L.MOE_ERR_UNSUPPORTED
    saved = L.MoeFfnSaved(16, 16, 16, 16)
    assert L.lib().moe_expert_ffn_save(cfg, None, 16, 16, ctypes.byref(_weights(cfg)), 16, 16, 16, ctypes.byref(saved), 16,
                                       BIG, 0, None) == L.MOE_ERR_UNSUPPORTED


def test_binding_refuses_host_and_strided_tensors():
    t = torch.zeros((4, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.moe_quantize_int8(t, 1, 4, 16, 1, 16, 16, stream=0)
    with pytest.raises(ValueError):
        L.moe_quantize_int8(t.t(), 1, 16, 4, 1, 16, 16, stream=0)
