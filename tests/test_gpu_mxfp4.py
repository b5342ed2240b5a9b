"""GPU parity of the MXFP4 path (E2M1 codes, one power of two per 32 elements).

Quantisation and reading back are exact on both sides, so codes, scale bytes and
values are compared bit for bit: every bf16 value, every (code, scale byte) pair,
special blocks, odd row counts, the quantising dispatch.  The expert GEMMs are
compared in two steps with a model in 64 bits: h before its quantisation from the
MXFP4 x and weights, and y from the GPU's own h.

Bounds (fixed before the first run).  A 128-wide K step is one MFMA: its products
are exact, their sum may be off by EPS_MFMA of the step's largest product (the
block-scaled MFMA of this chip aligns a step's products to the largest with a
limited width; 2^-10 is the allowance of the 8-bit tests), and the accumulator is
rounded once a step.  The sigmoid's exponential is off by about |g| 2^-24 plus a
few roundings.  y is rounded once to bf16 (2^-8 of the value at most)."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU, to_device
from gpu_util import dev_f32, dev_i32, host, say
from oracle import mxfp4 as mx
from workloads import MID
from workloads.inputs import f32_to_bf16_bits, make_weights, make_x, rng

pytestmark = pytest.mark.gpu

EPS_MFMA = 2.0 ** -10
EPS32 = 2.0 ** -24


def _quant_gpu(bits):
    """bf16 bit patterns [n, R, K] -> the oracle's form of the GPU's codes and scale bytes, per matrix."""
    n, R, K = bits.shape
    codes = torch.full((n, R, K // 2), 0xAA, dtype=torch.uint8, device="cuda")
    sc = torch.full((n, K // 128, R, 4), 0xAA, dtype=torch.uint8, device="cuda")
    L.moe_quantize_fp4(to_device(bits), n, R, K, codes, sc)
    torch.cuda.synchronize()
    return [mx.unpack(host(codes)[i], host(sc)[i]) for i in range(n)], codes, sc


def _check_quant(bits):
    got, codes, sc = _quant_gpu(bits)
    for i in range(bits.shape[0]):
        q, e = mx.quantize_mxfp4(oracle.decode_act(bits[i]))
        assert (got[i][1] == e).all()
        assert (got[i][0] == q).all()
    return codes, sc


# ---------------------------------------------------------------- quantisation, bit-exact
@pytest.mark.parametrize("top", [1.0, 1.75, 6.0, 2.0 ** -120, 2.0 ** -130, 3.3e38])
def test_quantize_every_bf16_value(top):
    """Every finite bf16 value of magnitude <= top, in blocks whose first element is top."""
    u = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    v = oracle.decode_act(u)
    tb = f32_to_bf16_bits(np.float32(top))
    vals = u[np.isfinite(v) & (np.abs(v) <= oracle.decode_act(tb[None] if tb.ndim else np.array([tb]))[0])]
    nb = -(-len(vals) // 31)
    nb += -nb % 4
    body = np.concatenate([vals, np.zeros(nb * 31 - len(vals), np.uint16)]).reshape(nb, 31)
    blocks = np.concatenate([np.full((nb, 1), tb, np.uint16), body], axis=1)
    say(f"mxfp4 sweep below {top}: {len(vals)} values")
    _check_quant(blocks.reshape(1, nb // 4, 128))


@pytest.mark.parametrize("n,R,K", [(1, 1, 128), (1, 1, 7168), (3, 37, 384), (2, 64, 1408), (1, 65, 2048), (5, 130, 128)])
def test_quantize_shapes(n, R, K):
    g = rng(61, n, R, K)
    x = g.standard_normal((n, R, K)).astype(np.float32) * np.exp2(g.integers(-20, 20, (n, R, K // 32))).repeat(32, -1)
    x[0, 0, :32] = 0
    say(f"mxfp4 quantize {n}x{R}x{K}")
    bits = f32_to_bf16_bits(x.astype(np.float32))
    codes, sc = _check_quant(bits)
    out = torch.empty((n, R, K), dtype=torch.bfloat16, device="cuda")
    L.moe_dequantize_fp4(codes, sc, n, R, K, out)
    torch.cuda.synchronize()
    for i in range(n):
        assert (host(out)[i] == mx.dequantize_mxfp4(*mx.quantize_mxfp4(oracle.decode_act(bits[i])))).all()


def test_quantize_special_blocks():
    x = np.ones((3, 256), np.float32)
    x[0, 3], x[0, 40], x[1, 200], x[2, 128:160] = np.nan, np.inf, -np.inf, 0
    x[1, 0] = -0.0
    bits = f32_to_bf16_bits(np.where(np.isnan(x), np.float32(1), x))[None].copy()
    bits[0, 0, 3] = 0x7FC1
    say("mxfp4 special blocks")
    codes, sc = _check_quant(bits)
    out = torch.empty((1, 3, 256), dtype=torch.bfloat16, device="cuda")
    L.moe_dequantize_fp4(codes, sc, 1, 3, 256, out)
    torch.cuda.synchronize()
    o = host(out)[0]
    assert np.isnan(o[0, :64]).all() and np.isnan(o[1, 192:224]).all() and (o[2, 128:160] == 0).all()
    assert np.isfinite(o).sum() == 3 * 256 - 96


def test_dequantize_every_code_and_scale():
    """All 16 codes under all 256 scale bytes; magnitudes from 2^128 up become infinite."""
    q = np.tile(np.arange(16, dtype=np.uint8), (256, 8))
    e = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    packed, sc = mx.pack(q, e)
    out = torch.empty((256, 128), dtype=torch.bfloat16, device="cuda")
    say("mxfp4 every code and scale byte")
    L.moe_dequantize_fp4(torch.from_numpy(packed).cuda(), torch.from_numpy(sc).cuda(), 1, 256, 128, out)
    torch.cuda.synchronize()
    want = mx.dequantize_mxfp4(q, e)
    want[np.abs(want) >= 2.0 ** 128] *= np.inf
    np.testing.assert_array_equal(host(out).astype(np.float64), want)


@pytest.mark.parametrize("T,H,k,noalloc", [(700, 384, 4, False), (1, 128, 1, False), (257, 7168, 3, True)])
def test_dispatch_mxfp4_exact(T, H, k, noalloc):
    E = 16
    cfg = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 1.0, "bf16", "mxfp4")
    g = rng(62, T, H)
    idx = np.argsort(-g.random((T, E)), axis=1)[:, :k].astype(np.int32)
    xb = f32_to_bf16_bits((g.standard_normal((T, H)) * np.exp(g.uniform(-6, 6, (T, 1)))).astype(np.float32))
    P = T * k
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(P), i32(T, k)
    xq = torch.empty((P, H // 2), dtype=torch.uint8, device="cuda")
    xs = torch.empty((H // 128, P, 4), dtype=torch.uint8, device="cuda")
    say(f"mxfp4 dispatch T={T} H={H} k={k} noalloc={noalloc}")
    args = (cfg, dev_i32(idx), to_device(xb), counts, offsets, perm, inv, xq, xs)
    if noalloc:
        L.moe_dispatch_noalloc(*args)
    else:
        L.moe_dispatch(*args, torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_DISPATCH), dtype=torch.uint8,
                                          device="cuda"))
    torch.cuda.synchronize()
    _, off_o, perm_o, inv_o = oracle.dispatch(idx, E)
    assert (host(perm) == perm_o).all() and (host(inv) == inv_o).all() and (host(offsets) == off_o).all()
    q, e = mx.quantize_mxfp4(oracle.decode_act(xb))
    gq, ge = mx.unpack(host(xq), host(xs))
    assert (gq == q[perm_o // k]).all() and (ge == e[perm_o // k]).all()


# ---------------------------------------------------------------- expert GEMMs on given routing
def _product(a, w):
    """a [R, K], w [N, K] MXFP4 values: the product in 64 bits and the bound on the GPU's."""
    R, K = a.shape
    out = a @ w.T
    aa, aw = np.abs(a), np.abs(w)
    bound = (K // 128 + 1) * EPS32 * (aa @ aw.T)
    for c in range(K // 128):
        ac, wc = aa[:, c * 128:(c + 1) * 128], aw[:, c * 128:(c + 1) * 128]
        for r0 in range(0, R, 16):
            bound[r0:r0 + 16] += EPS_MFMA * (ac[r0:r0 + 16, None, :] * wc[None]).max(axis=2)
    return out, bound


def _check_h(xq, wgu, hq, he):
    """GPU codes hq [R, I] and scale bytes he of h against h in 64 bits: every scale byte is that of an
    h within the bounds, every code the rounding of one."""
    I = wgu.shape[0] // 2
    (g, dg), (u, du) = _product(xq, wgu[:I]), _product(xq, wgu[I:])
    s = 1 / (1 + np.exp(-g))
    h = g * s * u
    # |d silu / dg| <= 1.1; the sigmoid's own error and three fp32 products
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(g * s) * du + (8 + np.abs(g)) * 2 * EPS32 * np.abs(h)
    R = h.shape[0]
    hb, db = h.reshape(R, I // 32, 32), dh.reshape(R, I // 32, 32)
    a = np.abs(hb)
    lo, hi = np.maximum(a - db, 0).max(axis=2), (a + db).max(axis=2)
    assert (mx.scale_byte(lo) <= he).all() and (he <= mx.scale_byte(hi)).all()
    x = np.exp2(he.astype(np.float64) - 127)[:, :, None]
    got = mx.e2m1_decode(hq).reshape(R, I // 32, 32)
    low, high = (hb - db) / x, (hb + db) / x
    assert (mx.e2m1_decode(mx.e2m1_encode(low)) <= got).all() and (got <= mx.e2m1_decode(mx.e2m1_encode(high))).all()
    q, e = mx.quantize_mxfp4(h)
    return float(((q == hq) | (mx.e2m1_decode(q) == mx.e2m1_decode(hq))).mean())


def _check_y(y, parts):
    """bf16 y against the sum of products of the GPU's own h: parts is a list of (h values, W_d values)."""
    want, bound = 0.0, 0.0
    for hv, wd in parts:
        p, b = _product(hv, wd)
        want, bound = want + p, bound + b + (len(parts) - 1) * EPS32 * (np.abs(hv) @ np.abs(wd).T)
    bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    assert (np.abs(y - want) <= bound + 1e-37).all(), float(np.abs(y - want).max())


def _part(layer, part, R, K):
    off, nb = L.moe_ffn_workspace_part(layer.cfg, part)
    n = R * K // 2
    codes = host(layer.ws_ffn[off:off + n].view(R, K // 2))
    off, nb = L.moe_ffn_workspace_part(layer.cfg, part + 1)
    return mx.unpack(codes, host(layer.ws_ffn[off:off + R * K // 32].view(K // 128, R, 4)))


def _spread(bits, g):
    """Every 32 elements times their own power of two in [2^-3, 2^3]: a scale applied to the wrong block,
    row or K step shows up as a large error."""
    v = oracle.decode_act(bits)
    f = np.exp2(g.integers(-3, 4, v.shape[:-1] + (v.shape[-1] // 32,))).repeat(32, -1)
    return f32_to_bf16_bits((v * f).astype(np.float32))


CASES = [
    # (T, H, E, G, M, k, S, I): tiles of 32 rows (up to 20 rows an expert on average) and of 128 and more, odd
    # numbers of 128-wide K steps in either GEMM, one step only, several shared experts, ragged tiles, one token,
    # more experts than pairs, column tiles past the end
    (1, 256, 8, 2, 1, 2, 1, 128),
    (1, 128, 4, 1, 1, 1, 0, 128),
    (64, 512, 4, 4, 4, 4, 0, 384),
    (33, 384, 64, 8, 3, 6, 3, 128),
    (300, 256, 8, 2, 2, 2, 1, 256),
    (517, 384, 16, 4, 2, 4, 2, 384),
    (300, 128, 4, 2, 2, 3, 3, 640),
    (1000, 1152, 8, 8, 3, 2, 2, 256),
    (130, 7168, 4, 2, 1, 2, 1, 128),
    (90, 256, 4, 1, 1, 2, 1, 2048),
    (100, 1152, 8, 2, 2, 3, 2, 384),
    (400, 256, 16, 4, 2, 2, 3, 128),
    # every routed segment as long as the batch: 256-row tiles, 288-row ones
    (288, 256, 2, 1, 1, 2, 1, 256),
    (577, 128, 1, 1, 1, 1, 2, 384),
    (250, 256, 2, 1, 1, 2, 1, 384),
    (240, 128, 2, 1, 1, 2, 1, 128),
    (500, 640, 2, 1, 1, 2, 3, 384),
    (560, 640, 2, 1, 1, 2, 3, 384),
    (270, 128, 2, 1, 1, 2, 1, 128),
    # 128-row tiles: tiles of one K step, more tiles than workgroups, shared experts' K ranges
    (100, 128, 4, 1, 1, 2, 1, 128),
    (700, 128, 24, 2, 2, 3, 2, 2048),
    (260, 1408, 12, 3, 3, 4, 3, 384),
]


def _layer(T, H, E, G, M, k, S, I, gather=False):
    c = MID.with_(T=T, H=H, E=E, G=G, M=M, k=k, S=S, I=I, sigma=0.05, group_topr=min(2, E // G), wgt="mxfp4")
    wts = make_weights(c)
    g = rng(63, T, H, E, S, I)
    wts.w_gate_up, wts.w_down = _spread(wts.w_gate_up, g), _spread(wts.w_down, g)
    if S:
        wts.ws_gate_up, wts.ws_down = _spread(wts.ws_gate_up, g), _spread(wts.ws_down, g)
    return c, wts, _spread(make_x(c), g), MoeLayerGPU(c, wts, gather=gather)


def _values(bits):
    return mx.dequantize_mxfp4(*mx.quantize_mxfp4(oracle.decode_act(bits)))


@pytest.mark.parametrize("T,H,E,G,M,k,S,I", CASES)
def test_expert_ffn_mxfp4(T, H, E, G, M, k, S, I):
    say(f"ffn mxfp4 T={T} H={H} E={E} k={k} S={S} I={I}")
    c, wts, xb, layer = _layer(T, H, E, G, M, k, S, I)
    bias = dev_f32(wts.bias0)
    y = layer.forward(to_device(xb), bias)
    torch.cuda.synchronize()
    offsets, tok = host(layer.offsets), host(layer.perm) // k
    xq = _values(xb)
    hq, he = _part(layer, L.MOE_WSP_H, T * k, I)
    hv = mx.dequantize_mxfp4(hq, he)
    yp = host(layer.y_perm)
    same = []
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        same.append(_check_h(xq[tok[a:b]], _values(wts.w_gate_up[e]), hq[a:b], he[a:b]))
        _check_y(yp[a:b], [(hv[a:b], _values(wts.w_down[e]))])
    if S:
        hq, he = _part(layer, L.MOE_WSP_H_SHARED, T, S * I)
        parts = []
        for s in range(S):
            cs, es = slice(s * I, (s + 1) * I), slice(s * I // 32, (s + 1) * I // 32)
            same.append(_check_h(xq, _values(wts.ws_gate_up[s]), hq[:, cs], he[:, es]))
            parts.append((mx.dequantize_mxfp4(hq[:, cs], he[:, es]), _values(wts.ws_down[s])))
        _check_y(host(layer.y_shared), parts)
    say(f"  h codes equal to the model's: {min(same):.6f}")
    assert np.isfinite(host(y)).all()


@pytest.mark.parametrize("T,H,E,G,M,k,S,I", [CASES[0], CASES[3], CASES[5], CASES[10], *CASES[-5:]])
def test_gather_and_phases_equal_sorted(T, H, E, G, M, k, S, I):
    """Rows gathered from x, and the two phases called apart, give the same bits as the whole call on sorted
    rows; rows that no pair has stay as they were."""
    c, wts, xb, layer = _layer(T, H, E, G, M, k, S, I)
    say(f"mxfp4 gather, phases T={T}")
    x, bias = to_device(xb), dev_f32(wts.bias0)
    layer.forward(x, bias)
    want = [layer.y_perm.clone(), layer.y_shared.clone() if S else None]
    for phases, gather in (((L.MOE_FFN_ALL,), True), ((L.MOE_FFN_GATE_UP, L.MOE_FFN_DOWN), False),
                           ((L.MOE_FFN_GATE_UP, L.MOE_FFN_DOWN), True)):
        layer.y_perm.fill_(float("nan"))
        layer.ws_ffn.fill_(0xFF)
        for ph in phases:
            if gather:
                L.moe_expert_ffn_gather(layer.cfg, x, layer.perm, layer.offsets, layer.weights, layer.y_perm,
                                        layer.y_shared, layer.ws_ffn, ph)
            else:
                layer.expert_ffn(x, ph)
        torch.cuda.synchronize()
        assert torch.equal(layer.y_perm.view(torch.int16), want[0].view(torch.int16))
        if S:
            assert torch.equal(layer.y_shared.view(torch.int16), want[1].view(torch.int16))


@pytest.mark.parametrize("i", [3, 5])
def test_layer_mxfp4_matches_oracle(i):
    """The whole layer against the oracle's, routing teacher-forced: a code of h can differ where h falls
    next to a rounding border, so the outputs are compared normwise (an E2M1 step is a quarter of the value
    and one of I codes of a row: well below 6e-2 of the largest output)."""
    c, wts, xb, layer = _layer(*CASES[i])
    say(f"mxfp4 layer {CASES[i]}")
    layer.forward(to_device(xb), dev_f32(wts.bias0))
    torch.cuda.synchronize()
    ref = oracle.layer_forward(c, xb, wts, wts.bias0, scores_in=host(layer.scores))
    assert (host(layer.topk_idx) == ref["idx"]).all()
    err = np.abs(host(layer.y).astype(np.float64) - ref["y"]).max() / np.abs(ref["y"]).max()
    say(f"  y err {err:.2e}")
    assert err < 6e-2


@pytest.mark.parametrize("i,gather", [(3, True), (5, False)])
def test_layer_mxfp4_graph_replays(i, gather):
    c, wts, xb, eager = _layer(*CASES[i], gather=gather)
    graph = MoeLayerGPU(c, wts, gather=gather)
    be, bg = dev_f32(wts.bias0), dev_f32(wts.bias0)
    xg = to_device(xb)
    say(f"mxfp4 graph {CASES[i]} gather={gather}")
    graph.capture(xg, bg, gamma=c.gamma)
    for step in range(4):
        xs = to_device(make_x(c, step))
        xg.copy_(xs)
        y = eager.forward(xs, be, gamma=c.gamma)
        torch.cuda.synchronize()
        yg = graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), yg.view(torch.int16)) and torch.equal(be, bg), step


def test_nan_block_reaches_its_rows_only():
    """A NaN in one token's x makes that token's outputs NaN and no other's."""
    c, wts, xb, layer = _layer(*CASES[5])
    xb = xb.copy()
    xb[7, 40] = 0x7FC0
    layer.scores.copy_(dev_f32(rng(64, 1).random((c.T, c.E)).astype(np.float32)))
    say("mxfp4 NaN row")
    layer.forward(to_device(xb), dev_f32(wts.bias0), scores_in=True)
    torch.cuda.synchronize()
    y = host(layer.y)
    assert np.isnan(y[7]).all() and np.isfinite(np.delete(y, 7, axis=0)).all()
