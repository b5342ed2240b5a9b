"""GPU tests of the share calls: dispatch, combine and their gradients where some (token,
slot) pairs are absent (experts held elsewhere, tokens behind the live ones, invalid ids).

Index outputs and copied rows are exact.  Sums are compared with 64-bit sums of the same
inputs: n terms added in fp32 are off by at most n 2^-24 of the sum of magnitudes, and
a bf16 result by another 2^-8 of its value (half a step), fp32 by 2^-24."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU, to_device
from gpu_util import dev_f32, dev_i32, host, say
from oracle import mxfp4 as mx
from workloads import MID, TINY
from workloads.inputs import f32_to_bf16_bits, make_weights, make_x, rng

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")
EPS32, BF = 2.0 ** -24, 2.0 ** -8


def _cfg(T, H, E, k, S=0, act="bf16", wgt=None):
    return L.make_cfg(T, H, E, 1, 1, k, S, 128, 1, 1.0, act, wgt or act)


def _sorted(idx, first, E, n):
    """The present pairs by brute force: counts, offsets, perm, inv."""
    T, k = idx.shape
    lists = [[] for _ in range(E)]
    for t in range(min(max(n, 0), T)):
        for j in range(k):
            e = int(idx[t, j]) - first
            if 0 <= e < E:
                lists[e].append(t * k + j)
    counts = np.array([len(v) for v in lists], np.int32)
    perm = np.array([f for v in lists for f in v], np.int32)
    inv = np.full(T * k, -1, np.int32)
    inv[perm] = np.arange(len(perm))
    return counts, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), perm, inv.reshape(T, k)


def _ids(T, total, k, seed, odd=True):
    """Expert ids with duplicates and ids of no expert among them."""
    g = rng(71, T, total, k, seed)
    idx = g.integers(0, total, (T, k)).astype(np.int32)
    if odd and T > 3:
        idx[0] = -1
        idx[1, 0], idx[2, 0], idx[3, 0] = -2 ** 31, 2 ** 31 - 1, total
    return idx


def _dispatch(cfg, first, n, idx, x, xp=None, xs=None):
    P, E = cfg.T * cfg.k, cfg.E
    out = [torch.full(s, -7, **I32) for s in ((E,), (E + 1,), (P,), (cfg.T, cfg.k))]
    ws = torch.full((L.moe_workspace_bytes(cfg, L.MOE_WS_DISPATCH),), 0xFF, dtype=torch.uint8, device="cuda")
    L.moe_dispatch_local(cfg, first, n, idx, x, *out, xp, xs, ws)
    torch.cuda.synchronize()
    return out


CASES = [
    # (T, H, total, first, E, k, n): one token; none; a part; every expert; windows at either end; live tokens
    # past T and below 0; more pairs than one segment; E no power of two; k past 8
    (1, 64, 4, 0, 4, 1, None),
    (1, 128, 4, 2, 2, 2, 0),
    (0, 64, 4, 0, 4, 2, None),
    (33, 192, 16, 4, 8, 3, 20),
    (257, 64, 256, 224, 32, 8, 999),
    (700, 320, 40, 13, 27, 6, 699),
    (1100, 128, 64, 0, 64, 2, -3),
    (5000, 64, 256, 0, 256, 8, 4001),
    (512, 128, 512, 0, 512, 8, 512),       # 4096 pairs: the last that one launch sorts
    (513, 128, 512, 5, 300, 8, 500),
    (130, 8320, 512, 100, 300, 32, 77),
    (4200, 64, 4, 1, 1, 1, None),
    (20000, 64, 256, 0, 256, 8, 19000),    # more segment counts than a workgroup adds up
]


@pytest.mark.parametrize("T,H,total,first,E,k,n", CASES)
@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8_e4m3", "mxfp4", "index"])
def test_dispatch_local_exact(T, H, total, first, E, k, n, kind):
    if kind in ("fp8_e4m3", "mxfp4"):
        H = max(128, H // 128 * 128) if kind == "mxfp4" or H <= 8192 else 8192
    act = "f32" if kind == "f32" else "bf16"
    wgt = kind if kind != "index" else "bf16"
    cfg = _cfg(T, H, E, k, act=act, wgt=wgt)
    idx = _ids(T, total, k, H)
    g = rng(72, T, H)
    xf = g.standard_normal((T, H)).astype(np.float32)
    xb = xf if act == "f32" else f32_to_bf16_bits(xf)
    P = T * k
    say(f"dispatch_local {kind} T={T} H={H} experts {first}+{E} of {total} k={k} n={n}")
    xp = xs = None
    if kind == "fp8_e4m3":
        xp = torch.full((P, H), 0x55, dtype=torch.uint8, device="cuda")
        xs = torch.full((P, H // 128), -5.0, device="cuda")
    elif kind == "mxfp4":
        xp = torch.full((P, H // 2), 0x55, dtype=torch.uint8, device="cuda")
        xs = torch.full((H // 128, P, 4), 0x55, dtype=torch.uint8, device="cuda")
    elif kind != "index":
        xp = torch.full((P, H), -5.0, dtype=torch.float32 if act == "f32" else torch.bfloat16, device="cuda")
    nt = None if n is None else torch.tensor([n], **I32)
    out = _dispatch(cfg, first, nt, dev_i32(idx), to_device(xb) if xp is not None else None, xp, xs)
    counts, offsets, perm, inv = (host(o) for o in out)
    wc, wo, wp, wi = _sorted(idx, first, E, T if n is None else n)
    m = len(wp)
    assert (counts == wc).all() and (offsets == wo).all() and (inv == wi).all()
    assert (perm[:m] == wp).all() and (perm[m:] == -7).all()
    tok = wp // k
    if kind == "mxfp4":
        q, e = mx.pack(*mx.quantize_mxfp4(oracle.decode_act(xb)[tok])) if m else (0, 0)
        assert (host(xp)[:m] == q).all() and (host(xs)[:, :m] == e).all()
        assert (host(xp)[m:] == 0x55).all() and (host(xs)[:, m:] == 0x55).all()
    elif kind == "fp8_e4m3":
        if m:
            q, s = oracle.quantize_rows_1x128(oracle.decode_act(xb)[tok])
            assert (host(xp)[:m] == q).all() and (host(xs)[:m] == s).all()
        assert (host(xp)[m:] == 0x55).all() and (host(xs)[m:] == -5).all()
    elif xp is not None:
        assert (host(xp)[:m] == oracle.decode_act(xb)[tok]).all() and (host(xp)[m:] == -5).all()


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (500, 64, 6), (2000, 256, 8)])
def test_whole_batch_equals_plain_calls(T, E, k):
    """With every pair present the share calls give the plain calls' bits."""
    H, S = 256, 1
    cfg = _cfg(T, H, E, k, S)
    g = rng(73, T, E)
    idx = dev_i32(np.argsort(g.random((T, E)), axis=1)[:, :k])
    bf = lambda *s: to_device(f32_to_bf16_bits(g.standard_normal(s).astype(np.float32)))
    x, yp, ys, dy, dxp, dxs = bf(T, H), bf(T * k, H), bf(T, H), bf(T, H), bf(T * k, H), bf(T, H)
    w, dxr = dev_f32(g.random((T, k))), dev_f32(g.standard_normal((T, H)))
    say(f"share calls over a whole batch T={T} E={E} k={k}")
    ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_DISPATCH), dtype=torch.uint8, device="cuda")
    got = []
    for local in (False, True):
        o = [torch.empty(s, **I32) for s in ((E,), (E + 1,), (T * k,), (T, k))]
        z = [torch.empty_like(yp), torch.empty_like(x), torch.empty_like(yp), torch.empty_like(w), torch.empty_like(x)]
        if local:
            L.moe_dispatch_local(cfg, 0, None, idx, x, *o, z[0], None, ws)
            L.moe_combine_local(cfg, yp, ys, o[3], w, z[1])
            L.moe_combine_local_backward(cfg, dy, yp, o[3], w, z[2], z[3])
            L.moe_dispatch_local_backward(cfg, dxp, dxs, dxr, o[3], z[4])
        else:
            L.moe_dispatch(cfg, idx, x, *o, z[0], None, ws)
            L.moe_combine(cfg, yp, ys, o[3], w, z[1])
            L.moe_combine_backward(cfg, dy, yp, o[3], w, z[2], z[3])
            L.moe_dispatch_backward(cfg, dxp, dxs, dxr, o[3], z[4])
        torch.cuda.synchronize()
        got.append(o + z)
    for i, (a, b) in enumerate(zip(*got)):
        if i == 7:   # d_topk_w: the same products, summed in another order
            assert ((a - b).abs() <= 2 * H * EPS32 * (H * 16.0)).all()
        else:
            assert torch.equal(a, b), i


SUMS = [
    # (T, H, total, first, E, k, n, S)
    (1, 64, 4, 0, 4, 1, None, 0),
    (1, 128, 4, 4, 4, 2, None, 1),
    (40, 64, 16, 4, 8, 3, 20, 1),
    (300, 7168, 64, 8, 8, 8, 280, 0),
    (65, 8320, 64, 0, 48, 32, None, 1),
    (200, 1344, 16, 0, 16, 5, 0, 0),
]


def _share(T, H, total, first, E, k, n, S, seed, act="bf16"):
    """A share's inputs; rows behind the last present pair and gates of absent slots are NaN."""
    cfg = _cfg(T, H, E, k, S, act)
    idx = _ids(T, total, k, seed, odd=False)
    _, _, perm, inv = _sorted(idx, first, E, T if n is None else n)
    g = rng(74, T, H, seed)
    m = len(perm)

    def rows(r, tail=False):
        v = g.standard_normal((r, H)).astype(np.float32)
        if tail:
            v[m:] = np.nan
        return v if act == "f32" else _bits_nan(v)

    w = (0.1 + g.random((T, k))).astype(np.float32)
    w[inv < 0] = np.nan
    return cfg, inv, m, w, rows


def _bits_nan(v):
    b = f32_to_bf16_bits(np.nan_to_num(v))
    b[np.isnan(v)] = 0x7FC0
    return b


def _val(a):
    return oracle.decode_act(a).astype(np.float64)


@pytest.mark.parametrize("T,H,total,first,E,k,n,S", SUMS)
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_combine_local(T, H, total, first, E, k, n, S, act):
    cfg, inv, m, w, rows = _share(T, H, total, first, E, k, n, S, 1, act)
    yp, ys = rows(T * k, True), rows(T) if S else None
    say(f"combine_local {act} T={T} H={H} experts {first}+{E} of {total} k={k} n={n} S={S}")
    y = torch.full((T, H), 9.0, dtype=torch.float32 if act == "f32" else torch.bfloat16, device="cuda")
    L.moe_combine_local(cfg, to_device(yp), to_device(ys), dev_i32(inv), dev_f32(w), y)
    torch.cuda.synchronize()
    here = (inv >= 0)[:, :, None]
    terms = np.where(here, np.nan_to_num(_val(yp))[np.maximum(inv, 0)] * np.nan_to_num(w).astype(np.float64)[:, :, None], 0)
    want, mag = terms.sum(1), np.abs(terms).sum(1)
    if S:
        want, mag = want + _val(ys), mag + np.abs(_val(ys))
    tol = (k + 2) * EPS32 * mag
    tol = tol + (BF if act == "bf16" else EPS32) * (np.abs(want) + tol)
    got = host(y).astype(np.float64)
    assert (np.abs(got - want) <= tol).all()
    if not S:
        assert (got[~here.any(axis=(1, 2))] == 0).all()


@pytest.mark.parametrize("T,H,total,first,E,k,n,S", SUMS)
@pytest.mark.parametrize("router", [True, False])
def test_backward_local(T, H, total, first, E, k, n, S, router):
    cfg, inv, m, w, rows = _share(T, H, total, first, E, k, n, S, 2)
    dy, yp, dxp, dxs = rows(T), rows(T * k, True), rows(T * k, True), rows(T) if S else None
    dxr = rng(75, T).standard_normal((T, H)).astype(np.float32) if router else None
    say(f"backward_local T={T} H={H} experts {first}+{E} of {total} k={k} n={n} S={S} router={router}")
    dyp = torch.full((T * k, H), 3.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), 3.0, device="cuda")
    dx = torch.full((T, H), 3.0, dtype=torch.bfloat16, device="cuda")
    d_inv = dev_i32(inv)
    L.moe_combine_local_backward(cfg, to_device(dy), to_device(yp), d_inv, dev_f32(w), dyp, dw)
    L.moe_dispatch_local_backward(cfg, to_device(dxp), to_device(dxs), None if dxr is None else dev_f32(dxr), d_inv, dx)
    torch.cuda.synchronize()
    here, rowi = inv >= 0, np.maximum(inv, 0)
    v_dy, v_yp, v_dxp = _val(dy), np.nan_to_num(_val(yp)), np.nan_to_num(_val(dxp))
    prod = v_dy[:, None, :] * v_yp[rowi]
    want, tol = prod.sum(2) * here, (H + 1) * EPS32 * np.abs(prod).sum(2)
    got = host(dw).astype(np.float64)
    assert (np.abs(got - want) <= tol).all() and (got[~here] == 0).all()
    full = np.full((T * k, H), 3.0)
    t, j = np.nonzero(here)
    full[inv[t, j]] = w[t, j].astype(np.float64)[:, None] * v_dy[t]
    assert (np.abs(host(dyp) - full) <= (BF + EPS32) * np.abs(full)).all()      # (an fp32 product, then bf16)
    assert (host(dyp)[m:] == 3).all()
    terms = np.where(here[:, :, None], v_dxp[rowi], 0)
    want, mag = terms.sum(1), np.abs(terms).sum(1)
    for extra in (None if dxs is None else _val(dxs), dxr):
        if extra is not None:
            want, mag = want + extra, mag + np.abs(extra)
    tol = (k + 3) * EPS32 * mag
    assert (np.abs(host(dx) - want) <= tol + BF * (np.abs(want) + tol)).all()


def test_gradients_against_differences():
    """Central differences of the fp32 forward calls: the step is linear in the gates, the expert outputs and
    the rows, so a difference over a step of 1 is the derivative itself up to fp32 rounding."""
    T, H, total, first, E, k, n = 24, 64, 12, 3, 6, 3, 20
    cfg, inv, m, w, rows = _share(T, H, total, first, E, k, n, 0, 3)
    f32 = _cfg(T, H, E, k, 0, "f32")
    w = np.nan_to_num(w, nan=0.5)
    dy, yp, gx = _val(rows(T)), np.nan_to_num(_val(rows(T * k, True))), np.nan_to_num(_val(rows(T * k, True)))
    bits = lambda v: to_device(f32_to_bf16_bits(v.astype(np.float32)))
    dyp, dw = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, k), device="cuda")
    dx = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    d_inv = dev_i32(inv)
    say("share gradients against differences")
    L.moe_combine_local_backward(cfg, bits(dy), bits(yp), d_inv, dev_f32(w), dyp, dw)
    L.moe_dispatch_local_backward(cfg, bits(gx), None, None, d_inv, dx)

    def combine(w_, yp_):
        y = torch.empty((T, H), device="cuda")
        L.moe_combine_local(f32, dev_f32(yp_), None, d_inv, dev_f32(w_), y)
        return host(y).astype(np.float64)

    mag = 16 * EPS32 * (k + 2) * (np.abs(dy).sum(1) * np.abs(yp).max() * 2 + 1)
    for j in range(k):
        hi, lo = w.copy(), w.copy()
        hi[:, j] += 0.5
        lo[:, j] -= 0.5
        diff = ((combine(hi, yp) - combine(lo, yp)) * dy).sum(1)
        assert (np.abs(diff - host(dw)[:, j]) <= mag + H * EPS32 * np.abs(dy).sum(1) * np.abs(yp).max()).all()
        at = inv[:, j][inv[:, j] >= 0]
        hi, lo = yp.copy(), yp.copy()
        hi[at] += 0.5
        lo[at] -= 0.5
        diff = (combine(w, hi) - combine(w, lo)) * dy
        have = inv[:, j] >= 0
        got = host(dyp)[at].astype(np.float64)
        assert (np.abs(diff[have] - got) <= BF * np.abs(got) + mag.max()).all()
    # x -> x_perm is a copy: <gx, x_perm(x + d)> - <gx, x_perm(x - d)> = sum over the present slots of gx
    idx = _ids(T, total, k, 3, odd=False)
    x = rng(76, 1).standard_normal((T, H)).astype(np.float32)
    outs = []
    for d in (0.5, -0.5):
        xp = torch.zeros((T * k, H), device="cuda")
        _dispatch(f32, first, torch.tensor([n], **I32), dev_i32(idx), dev_f32(x + np.float32(d)), xp)
        outs.append(host(xp).astype(np.float64) * gx)
    diff = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                diff[t] += (outs[0] - outs[1])[inv[t, j]]
    assert (np.abs(diff - host(dx)) <= BF * np.abs(diff) + 64 * EPS32 * (np.abs(gx).max() * 8 * k)).all()


# ---------------------------------------------------------------- a run of them together
RUNS = [
    ("f32", TINY.with_(T=96, k=3), 1e-5),
    ("bf16", MID.with_(T=300, H=256, E=16, G=4, M=2, k=4, S=1, I=256), 3 * BF),
    ("bf16 gather", MID.with_(T=300, H=256, E=16, G=4, M=2, k=4, S=0, I=256), 3 * BF),
    ("fp8", MID.with_(T=300, H=256, E=16, G=4, M=2, k=4, S=1, I=256, wgt="fp8_e4m3"), 3 * BF),
    ("mxfp4", MID.with_(T=300, H=256, E=16, G=4, M=2, k=4, S=1, I=256, wgt="mxfp4"), 3 * BF),
    ("mxfp4 gather", MID.with_(T=40, H=256, E=16, G=4, M=2, k=4, S=1, I=384, wgt="mxfp4"), 3 * BF),
    ("f32 gather", TINY.with_(T=96, k=3), 1e-5),
]


@pytest.mark.parametrize("label,c,tol", RUNS, ids=[r[0] for r in RUNS])
def test_shares_sum_to_the_layer(label, c, tol):
    """Three ranks' shares (the shared experts on the first) sum to the whole layer: every present pair's row
    is computed once, as in the whole layer, and only the rounding of each share's sum to the activation type
    is added (half a step of each of three partial sums and of the whole; for bf16 rows another half a step of
    each side, so 3 times 2^-8 of the magnitudes in all)."""
    gather = "gather" in label
    wts, xb = make_weights(c), make_x(c)
    x, bias = to_device(xb), dev_f32(wts.bias0)
    say(f"shares of {label}")
    whole = MoeLayerGPU(c, wts, gather=gather)
    y = host(whole.forward(x, bias)).astype(np.float64)
    offs, seen = host(whole.offsets), 0
    total, mag = np.zeros_like(y), np.zeros_like(y)
    cut = [0, 5, 9, 16]
    for r in range(3):
        cr = c if r == 0 else c.with_(S=0)
        layer = MoeLayerGPU(cr, wts, gather=gather, share=(cut[r], cut[r + 1] - cut[r]))
        for t in (layer.perm, layer.y_perm, layer.x_perm):
            if t is not None:
                t.view(torch.uint8).fill_(0xFF)      # what lies behind the present pairs must not matter
        layer.ws_ffn.fill_(0xFF)
        part = host(layer.forward(x, bias)).astype(np.float64)
        n = int(layer.offsets[-1])
        a = offs[cut[r]]
        assert n == offs[cut[r + 1]] - a
        got, want = layer.y_perm[:n].double(), whole.y_perm[a:a + n].double()
        if c.wgt == "bf16":
            # the bf16 down GEMM starts each tile's walk over K at a slice that depends on the tile's place in the
            # table: I products added in another order differ by 2 I 2^-24 of the sum of their magnitudes, at most
            # I max|h| max|w|, and both are then rounded to bf16
            off, _ = L.moe_ffn_workspace_part(layer.cfg_x, L.MOE_WSP_H)
            h = layer.ws_ffn[off:off + n * c.I * 2].view(torch.bfloat16).double().abs().max() if n else 0.0
            order = 2 * c.I * EPS32 * c.I * h * layer.w_down.double().abs().max()
            assert ((got - want).abs() <= order + 2 * BF * (want.abs() + order)).all()
        else:
            assert torch.equal(got, want)
        seen += n
        total, mag = total + part, mag + np.abs(part)
    assert seen == c.T * c.k
    assert (np.abs(total - y) <= tol * (mag + np.abs(y)) + 1e-30).all()


@pytest.mark.parametrize("wgt", ["bf16", "mxfp4"])
def test_padded_batch_replays(wgt):
    """A graph over a padded batch follows n_tokens from replay to replay, with an eager step's bits; live
    tokens come out as in the whole batch, padded ones with the shared experts' part alone."""
    c = MID.with_(T=200, H=256, E=16, G=4, M=2, k=4, S=1, I=256, wgt=wgt)
    wts = make_weights(c)
    bias = dev_f32(wts.bias0)
    eager, graph = MoeLayerGPU(c, wts), MoeLayerGPU(c, wts)
    xg, ng = to_device(make_x(c, 0)), torch.tensor([c.T], **I32)
    say(f"padded graph {wgt}")
    graph.capture(xg, bias, n_tokens=ng)
    for step, n in enumerate((200, 1, 0, 133)):
        xs = to_device(make_x(c, step))
        xg.copy_(xs)
        ng.fill_(n)
        whole = eager.forward(xs, bias).clone()
        y = eager.forward(xs, bias, n_tokens=torch.tensor([n], **I32)).clone()
        torch.cuda.synchronize()
        yg = graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), yg.view(torch.int16)), step
        assert int(graph.offsets[-1]) == n * c.k
        assert torch.equal(y[:n].view(torch.int16), whole[:n].view(torch.int16)), step
        assert torch.equal(y[n:], eager.y_shared[n:]), step


@pytest.mark.parametrize("gather", [True, False])
def test_live_rows_choose_the_mxfp4_tiles(gather):
    """One graph of a padded batch whose live rows an expert ask for 256-, 288- and 128-row tiles in turn: the same
    bits for a live token whatever the tiles (its products and sums have one order)."""
    c = MID.with_(T=1100, H=384, E=4, G=1, M=1, k=2, S=1, I=256, wgt="mxfp4")
    wts = make_weights(c)
    bias, x = dev_f32(wts.bias0), to_device(make_x(c))
    whole = MoeLayerGPU(c, wts, gather=gather)
    want = whole.forward(x, bias).clone()
    layer, n = MoeLayerGPU(c, wts, gather=gather), torch.tensor([c.T], **I32)
    say(f"tiles of live rows gather={gather}")
    layer.capture(x, bias, n_tokens=n)
    for live in (1100, 1000, 200, 5, 1000, 1100):
        n.fill_(live)
        layer.y.zero_()
        layer.y_perm.fill_(float("nan"))
        torch.cuda.synchronize()
        y = layer.replay()
        torch.cuda.synchronize()
        assert int(layer.offsets[-1]) == 2 * live
        assert torch.equal(y[:live].view(torch.int16), want[:live].view(torch.int16)), live
        assert torch.equal(y[live:].view(torch.int16), layer.y_shared[live:].view(torch.int16)), live


def test_training_step_of_a_share():
    """Forward and backward of two shares on buffers whose unused rows are NaN: the weight gradients are the
    whole layer's for the experts held, and dx and the router's gradient sum to the whole layer's."""
    c = MID.with_(T=260, H=256, E=16, G=4, M=2, k=4, S=1, I=256)
    wts, xb = make_weights(c), make_x(c)
    x, bias = to_device(xb), dev_f32(wts.bias0)
    dy = to_device(f32_to_bf16_bits(rng(77, 1).standard_normal((c.T, c.H)).astype(np.float32)))
    say("training step of shares")

    def step(layer):
        layer.forward(x, bias)
        layer.alloc_backward()
        for t in (layer.dy_perm, layer.dx_perm, layer.ws_ffn_bwd):
            t.view(torch.uint8).fill_(0xFF)
        dx = host(layer.backward(x, dy)).astype(np.float64)
        torch.cuda.synchronize()
        return dx, host(layer.g_w_router).astype(np.float64), host(layer.g_w_gate_up), host(layer.g_w_down)

    dx, gr, gu, gd = step(MoeLayerGPU(c, wts))
    sum_dx, sum_gr = 0.0, 0.0
    for r, (a, b) in enumerate(((0, 7), (7, 16))):
        layer = MoeLayerGPU(c if r == 0 else c.with_(S=0), wts, share=(a, b - a))
        for t in (layer.x_perm, layer.y_perm, layer.perm):
            t.view(torch.uint8).fill_(0xFF)
        dxr, grr, gur, gdr = step(layer)
        # the same rows in the same order through the same kernel
        assert np.abs(gur - gu[a:b]).max() <= 2.0 ** -16 * np.abs(gu).max()
        assert np.abs(gdr - gd[a:b]).max() <= 2.0 ** -16 * np.abs(gd).max()
        sum_dx, sum_gr = sum_dx + dxr, sum_gr + grr
    # each dx, and each dlogit in bf16 before the router's product, is rounded on its own
    assert np.abs(sum_dx - dx).max() <= 6 * BF * np.abs(dx).max()
    assert np.abs(sum_gr - gr).max() <= 6 * BF * np.abs(gr).max()
    with pytest.raises(ValueError):
        layer.n_tokens = torch.tensor([5], **I32)
        layer.backward(x, dy, alpha=0.1)


def test_two_streams_at_once():
    """Two shares of one batch on two streams, each with its own buffers, give what they give alone."""
    c = MID.with_(T=1500, H=512, E=32, G=4, M=2, k=4, S=0, I=256, wgt="mxfp4")
    wts = make_weights(c)
    x, bias = to_device(make_x(c)), dev_f32(wts.bias0)
    layers = [MoeLayerGPU(c, wts, share=s) for s in ((0, 16), (16, 16))]
    alone = [lay.forward(x, bias).clone() for lay in layers]
    torch.cuda.synchronize()
    say("two shares on two streams")
    streams = [torch.cuda.Stream() for _ in layers]
    for lay, st in zip(layers, streams):
        lay.y.zero_()
    torch.cuda.synchronize()
    for lay, st in zip(layers, streams):
        with torch.cuda.stream(st):
            lay.forward(x, bias)
    torch.cuda.synchronize()
    for lay, want in zip(layers, alone):
        assert torch.equal(lay.y.view(torch.int16), want.view(torch.int16))


def test_rows_past_32_bit_offsets():
    """A batch that repeats 512 tokens 128 times: its permuted rows take 7.5 GB, and every repetition gives what
    the 512 tokens give alone, bit for bit (a row's products and sums do not depend on where it lies)."""
    n, R, H, E, k = 512, 128, 7168, 8, 8
    g = rng(78, 1)
    c = MID.with_(T=n, H=H, E=E, G=1, M=1, k=k, S=1, I=128, sigma=0.05, wgt="mxfp4")
    wts = make_weights(c)
    bits = lambda *s: to_device(f32_to_bf16_bits(g.standard_normal(s).astype(np.float32)))
    x, dy = bits(n, H), bits(n, H)
    idx = dev_i32(np.argsort(g.random((n, E)), axis=1).astype(np.int32))
    w = dev_f32(g.random((n, k)).astype(np.float32))
    held = MoeLayerGPU(c, wts, T=1)          # its quantised weights

    def run(T):
        cfg = L.make_cfg(T, H, E, 1, 1, k, 1, 128, 1, 1.0, "bf16", "mxfp4")
        grad = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 1.0, "bf16", "bf16")
        rep = lambda a: a.repeat(T // n, 1)
        u8, bf = dict(dtype=torch.uint8, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        P = T * k
        xp, xs = torch.empty((P, H // 2), **u8), torch.empty((H // 128, P, 4), **u8)
        xt, wt, dyt = rep(x), rep(w), rep(dy)
        _, offsets, _, inv = _dispatch(cfg, 0, None, rep(idx), xt, xp, xs)
        assert (host(offsets) == np.arange(E + 1) * T).all()
        yp, ysh, y, dx = torch.empty((P, H), **bf), *(torch.empty((T, H), **bf) for _ in range(3))
        ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_FFN), **u8)
        L.moe_expert_ffn(cfg, xp, xs, offsets, held.weights, xt, yp, ysh, ws)
        L.moe_combine_local(cfg, yp, ysh, inv, wt, y)
        dyp, dw = torch.empty((P, H), **bf), torch.empty((T, k), dtype=torch.float32, device="cuda")
        L.moe_combine_local_backward(grad, dyt, yp, inv, wt, dyp, dw)
        L.moe_dispatch_local_backward(grad, dyp, None, None, inv, dx)
        torch.cuda.synchronize()
        return [a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32) for a in (y, dw, dx)]

    say("rows past 32-bit offsets")
    for name, one, many in zip(("y", "d_topk_w", "dx"), run(n), run(n * R)):
        assert torch.equal(many.view(R, n, -1), one.view(1, n, -1).expand(R, -1, -1)), name
