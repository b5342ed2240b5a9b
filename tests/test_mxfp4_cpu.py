"""MXFP4 without a GPU: pins of the oracle's format, and the host-side refusals of the
library's MXFP4 calls (checked before any device call)."""
import ctypes

import numpy as np
import pytest
import torch

from biased_top_routing_amd import _lib as L
from oracle import mxfp4 as mx
from workloads import MID
from workloads.inputs import rng

BIG = 1 << 40


# ---------------------------------------------------------------- the oracle's format
def test_e2m1_codes_by_enumeration():
    """Every code decodes to its definition (bias 1, subnormal .5) and encodes back."""
    for c in range(16):
        s, ex, m = c >> 3, (c >> 1) & 3, c & 1
        want = (m * 0.5 if ex == 0 else (1 + m / 2) * 2.0 ** (ex - 1)) * (-1 if s else 1)
        got = mx.e2m1_decode(np.array([c], np.uint8))[0]
        assert got == want and np.signbit(got) == bool(s)
        assert mx.e2m1_encode(np.array([got]))[0] == c


def test_e2m1_ties_and_neighbours():
    """Midpoints go to the even code; a little to either side goes to that side."""
    for lo in range(7):
        mid = (mx.MAGS[lo] + mx.MAGS[lo + 1]) / 2
        even = lo if lo % 2 == 0 else lo + 1
        assert list(mx.e2m1_encode(np.array([mid, np.nextafter(mid, 0), np.nextafter(mid, 9)]))) == [even, lo, lo + 1]
    assert (mx.e2m1_encode(np.array([6.5, 100.0])) == 7).all()


def test_scale_keeps_every_rounding_within_half_a_step():
    """Brute force over the largest magnitudes of one octave and their blocks' elements."""
    g = rng(41, 1)
    for top in np.concatenate([np.linspace(1, 2, 257), [1.75, np.nextafter(1.75, 1), 2 ** -126, 2 ** -130, 3e38]]):
        v = np.concatenate([[top], g.uniform(-top, top, 31)])[None]
        q, e = mx.quantize_mxfp4(v)
        x = 2.0 ** (float(e[0, 0]) - 127)
        a = np.abs(v[0]) / x
        assert a.max() < 7 and (e[0, 0] == 1 or a.max() >= 3.5)
        step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
        assert (np.abs(mx.dequantize_mxfp4(q, e)[0] - v[0]) <= step / 2 * x).all()


def test_special_blocks():
    v = np.ones((4, 64))
    v[0, 5], v[1, 40], v[2, 7], v[3, :32] = np.nan, np.inf, -np.inf, 0
    q, e = mx.quantize_mxfp4(v)
    d = mx.dequantize_mxfp4(q, e)
    assert list(e[0]) == [255, 125] and np.isnan(d[0, :32]).all() and (d[0, 32:] == 1).all()
    assert list(e[1]) == [125, 255] and list(e[2]) == [255, 125]
    assert list(e[3]) == [1, 125] and (d[3, :32] == 0).all()


def test_pack_round_trips():
    g = rng(42, 1)
    q, e = mx.quantize_mxfp4(g.standard_normal((5, 384)))
    packed, sc = mx.pack(q, e)
    assert packed.shape == (5, 192) and sc.shape == (3, 5, 4)
    assert packed[2, 7] == q[2, 14] | q[2, 15] << 4 and sc[1, 3, 2] == e[3, 6]
    q2, e2 = mx.unpack(packed, sc)
    assert (q2 == q).all() and (e2 == e).all()


# ---------------------------------------------------------------- refusals of the library
@pytest.mark.parametrize("args,status", [
    ((None, 1, 4, 128, 16, 16), L.MOE_ERR_NULL),
    ((16, 1, 4, 128, None, 16), L.MOE_ERR_NULL),
    ((16, 1, 4, 128, 16, None), L.MOE_ERR_NULL),
    ((16, -1, 4, 128, 16, 16), L.MOE_ERR_SHAPE),
    ((16, 1, -4, 128, 16, 16), L.MOE_ERR_SHAPE),
    ((16, 1, 4, 0, 16, 16), L.MOE_ERR_SHAPE),
    ((16, 1, 4, 96, 16, 16), L.MOE_ERR_SHAPE),
    ((16, 65536, 4, 128, 16, 16), L.MOE_ERR_SHAPE),
    ((16, 1, 2147483647, 128 * 64, 16, 16), L.MOE_ERR_SHAPE),
    ((16, 1, 1 << 28, 128, 16, 16), L.MOE_ERR_SHAPE),      # a grid of 2^32 lanes
    ((8, 1, 4, 128, 16, 16), L.MOE_ERR_UNSUPPORTED),       # misaligned
    ((16, 1, 4, 128, 18, 16), L.MOE_ERR_UNSUPPORTED),
    ((16, 1, 4, 128, 16, 17), L.MOE_ERR_UNSUPPORTED),
])
def test_quantize_refusals(args, status):
    src, n, rows, cols, codes, sc = args
    assert L.lib().moe_quantize_fp4(src, n, rows, cols, codes, sc, None) == status
    assert L.lib().moe_dequantize_fp4(codes, sc, n, rows, cols, src, None) == status


def test_quantize_nothing_is_ok():
    assert L.lib().moe_quantize_fp4(16, 0, 4, 128, 16, 16, None) == L.MOE_OK
    assert L.lib().moe_dequantize_fp4(16, 16, 3, 0, 128, 16, None) == L.MOE_OK


def test_binding_refuses_strided_tensors():
    x = torch.zeros((8, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((1, 8, 4), dtype=torch.uint8)
    with pytest.raises(ValueError):
        L.moe_quantize_fp4(x[:, ::2], 1, 8, 128, q, s, stream=0)
    with pytest.raises(ValueError):
        L.moe_dequantize_fp4(q.t(), s, 1, 64, 128, x, stream=0)


def _cfg(**kw):
    return L.cfg_from(MID, wgt="mxfp4", **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(H=2048 + 64), L.MOE_ERR_SHAPE),
    (dict(I=1408 + 64), L.MOE_ERR_SHAPE),
    (dict(act="f32"), L.MOE_ERR_UNSUPPORTED),
    (dict(T=1 << 23, H=2048, k=6), L.MOE_ERR_SHAPE),       # T*k*H past 2^36: 32-bit scale offsets
])
def test_config_refusals(kw, status):
    cfg = _cfg(**kw)
    assert L.moe_workspace_bytes(cfg, L.MOE_WS_FFN) == 0
    assert L.lib().moe_update_bias(ctypes.byref(cfg), 1, 1, 1e-3, None) == status


def test_ffn_refusals():
    cfg = _cfg()
    ok = (16,) * 8
    w = L.MoeExpertWeights(*ok)
    need = L.moe_workspace_bytes(cfg, L.MOE_WS_FFN)
    fn, fg = L.lib().moe_expert_ffn, L.lib().moe_expert_ffn_gather
    c = ctypes.byref(cfg)
    assert fn(c, 16, None, 16, ctypes.byref(w), 16, 16, 16, 16, need, 0, None) == L.MOE_ERR_NULL       # row scales
    assert fn(c, 16, 16, 16, ctypes.byref(w), 16, 16, 16, 16, need - 1, 0, None) == L.MOE_ERR_WORKSPACE
    for i in range(8):
        miss = L.MoeExpertWeights(*(None if j == i else 16 for j in range(8)))
        assert fn(c, 16, 16, 16, ctypes.byref(miss), 16, 16, 16, 16, need, 0, None) == L.MOE_ERR_NULL, i
        off = L.MoeExpertWeights(*(18 if j == i else 16 for j in range(8)))
        assert fn(c, 16, 16, 16, ctypes.byref(off), 16, 16, 16, 16, need, 0, None) == L.MOE_ERR_UNSUPPORTED, i
    assert fg(c, 24, 16, 16, ctypes.byref(w), 16, 16, 16, need, 0, None) == L.MOE_ERR_UNSUPPORTED     # x misaligned
    assert fg(c, 16, None, 16, ctypes.byref(w), 16, 16, 16, need, 0, None) == L.MOE_ERR_NULL
    # (T + 1) * H / 2 past 2^31 - 1
    wide = _cfg(T=1 << 21, H=2048, k=1, M=1)
    assert fg(ctypes.byref(wide), 16, 16, 16, ctypes.byref(w), 16, 16, 16, BIG, 0, None) == L.MOE_ERR_UNSUPPORTED
    save = L.MoeFfnSaved(16, 16, 16, 16)
    assert L.lib().moe_expert_ffn_save(c, 16, None, 16, ctypes.byref(w), 16, 16, 16, ctypes.byref(save), 16, need, 0,
                                       None) != L.MOE_OK                                              # bf16 only
    assert L.lib().moe_combine_backward(c, 16, 16, 16, 16, 16, 16, None) == L.MOE_ERR_UNSUPPORTED


def test_dispatch_refusals():
    cfg = _cfg()
    need = L.moe_workspace_bytes(cfg, L.MOE_WS_DISPATCH)
    fn = L.lib().moe_dispatch
    c = ctypes.byref(cfg)
    assert fn(c, 16, 16, 16, 16, 16, 16, 16, None, 16, need, None) == L.MOE_ERR_NULL
    assert fn(c, 16, 24, 16, 16, 16, 16, 16, 16, 16, need, None) == L.MOE_ERR_UNSUPPORTED
    assert fn(c, 16, 16, 16, 16, 16, 16, 24, 16, 16, need, None) == L.MOE_ERR_UNSUPPORTED
    assert fn(c, 16, 16, 16, 16, 16, 16, 16, 18, 16, need, None) == L.MOE_ERR_UNSUPPORTED


def test_workspace_parts():
    cfg = _cfg()
    total = L.moe_workspace_bytes(cfg, L.MOE_WS_FFN)
    P, T = MID.T * MID.k, MID.T
    want = [P * MID.I // 2, P * MID.I // 32, T * MID.S * MID.I // 2, T * MID.S * MID.I // 32]
    end = 0
    for part, n in enumerate(want):
        off, nb = L.moe_ffn_workspace_part(cfg, part)
        assert off >= end and nb >= n and off % 256 == 0
        end = off + nb
    assert end + T * MID.H * 17 // 32 <= total
