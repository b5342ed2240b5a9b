"""GPU parity of softmax routing and raw gates, and of their gradients.

Activations and router weights lie on grids that make every logit exact in fp32 whatever the order of its sum, so the
affinities (a softmax in 64 bits, rounded once) and the chosen experts are compared bit for bit with the oracle's.
Gates: a sum of at most 32 terms, a product and a quotient: 40 roundings of 2^-24.

Gradients (bounds fixed before the first run): dlogit is off by 100 2^-24 of the magnitudes that make it up and by 2^-17
of itself (two bf16 terms), a product over n terms adds n 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import to_device
from gpu_util import dev_f32, dev_i32, host, say
from workloads.inputs import f32_to_bf16_bits, rng

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24


def _inputs(T, H, E, act, seed=0):
    g = rng(121, T, H, E, seed)
    grid = lambda n, sigma, unit, most: (np.clip(np.rint(g.standard_normal((n, H)) * sigma / unit), -most, most) * unit
                                         ).astype(np.float32)
    x, w = grid(T, 1.0, 2.0 ** -3, 32), grid(E, 1.5 / np.sqrt(H), 2.0 ** -11, 61)
    return x, w, (g.uniform(-0.1, 0.1, E) / E).astype(np.float32)


ROUTE = [
    # (T, H, E, G, M, k, topr, act): one token, the split router kernels, the fused one, every tile of the large ones,
    # the general selection (E no multiple of 16, groups of odd sizes, k past 16)
    (1, 128, 16, 4, 2, 4, 2, "bf16"),
    (128, 7168, 256, 8, 4, 8, 2, "bf16"),
    (1500, 256, 256, 8, 4, 8, 2, "bf16"),
    (2049, 128, 256, 8, 4, 8, 3, "bf16"),
    (9000, 64, 128, 4, 4, 6, 1, "bf16"),
    (9000, 64, 64, 8, 3, 6, 2, "bf16"),
    (16384, 64, 256, 8, 4, 8, 4, "bf16"),
    (33000, 64, 256, 1, 1, 8, 1, "bf16"),
    (65537, 64, 256, 16, 4, 2, 2, "bf16"),
    (37, 192, 13, 1, 1, 5, 1, "bf16"),
    (300, 64, 60, 5, 3, 20, 5, "bf16"),
    (257, 64, 300, 3, 2, 32, 8, "bf16"),
    (9, 64, 512, 64, 7, 3, 2, "bf16"),
    (50, 64, 2, 2, 1, 1, 1, "bf16"),
    (65, 128, 16, 4, 2, 4, 2, "f32"),
    (33, 36, 7, 7, 3, 2, 1, "f32"),
    (3, 4, 1, 1, 1, 1, 1, "f32"),
]


def _route(cfg, x, w, o, bias, flags, keep):
    T, E, k = cfg.T, cfg.E, cfg.k
    s = torch.full((T, E), -3.0, device="cuda") if keep else None
    idx, gates = torch.full((T, k), -1, dtype=torch.int32, device="cuda"), torch.full((T, k), -1.0, device="cuda")
    ws = None if keep else torch.full((L.moe_workspace_bytes(cfg, L.MOE_WS_ROUTE),), 0xFF, dtype=torch.uint8, device="cuda")
    L.moe_route(cfg, x, w, o, bias, s, flags, idx, gates, ws)
    torch.cuda.synchronize()
    return None if s is None else host(s), host(idx), host(gates)


@pytest.mark.parametrize("mask", [None, "some"])
@pytest.mark.parametrize("T,H,E,G,M,k,topr,act", ROUTE)
def test_softmax_routing(T, H, E, G, M, k, topr, act, mask):
    say(f"softmax route T={T} H={H} E={E} G={G} M={M} k={k} {act} mask={mask}")
    x, w, bias = _inputs(T, H, E, act)
    o = None
    if mask:
        g = rng(122, E)
        o = g.standard_normal(E).astype(np.float32)
        o[g.random(E) < 0.2] = -np.inf
        o[g.random(E) < 0.1] = np.finfo(np.float32).min
    up = (lambda a: to_device(a)) if act == "f32" else (lambda a: to_device(f32_to_bf16_bits(a)))
    cfg = L.make_cfg(T, H, E, G, M, k, 0, 128, topr, 2.5, act, act)
    sr = oracle.affinity_softmax(x, w, o)
    for raw, keep in ((False, True), (True, False), (True, True), (False, False)):
        flags = L.MOE_SOFTMAX | (L.MOE_GATES_RAW if raw else 0)
        s, idx, gates = _route(cfg, up(x), up(w), None if o is None else dev_f32(o), dev_f32(bias), flags, keep)
        ir, gr = oracle.route(sr, bias, G, M, k, topr, 2.5, raw)
        if keep:
            assert (s == sr).all()
        assert (idx == ir).all()
        assert (np.abs(gates - gr) <= 40 * EPS32 * gr).all()


@pytest.mark.parametrize("T,E,G,k", [(9, 256, 8, 8), (2100, 256, 8, 8), (9, 64, 4, 6), (5000, 64, 4, 6), (9, 60, 5, 20)])
def test_a_row_with_a_nan_or_an_infinity(T, E, G, k):
    """Its affinities are NaN, its experts some of the E, and no other row changes."""
    x, w, bias = _inputs(T, 64, E, "bf16")
    cfg = L.make_cfg(T, 64, E, G, G, k, 0, 128, 2, 1.0, "bf16", "bf16")
    say(f"softmax of NaN T={T} E={E}")
    run = lambda a: _route(cfg, to_device(f32_to_bf16_bits(a)), to_device(f32_to_bf16_bits(w)), None, dev_f32(bias),
                           L.MOE_SOFTMAX, True)
    want = run(x)
    bad = x.copy()
    bad[1, 5], bad[T - 1, 0] = np.nan, np.inf
    s, idx, gates = run(bad)
    assert np.isnan(s[[1, T - 1]]).all() and np.isnan(gates[[1, T - 1]]).all() and (idx >= 0).all() and (idx < E).all()
    for got, ref in zip((s, idx, gates), want):
        rest = np.delete(np.arange(T), [1, T - 1])
        assert (got[rest] == ref[rest]).all()


@pytest.mark.parametrize("E,G,M,k,topr", [(256, 8, 4, 8, 2), (256, 1, 1, 16, 4), (128, 16, 3, 6, 1), (128, 2, 1, 1, 3),
                                          (256, 16, 16, 16, 4)])
@pytest.mark.parametrize("flags", [0, L.MOE_GATES_RAW])
def test_the_selection_of_a_token_does_not_depend_on_the_batch(E, G, M, k, topr, flags):
    """Few tokens are selected by a wavefront each, many by 16 lanes each: the same experts and gates, bit for bit, with
    ties, affinities of zero and masked experts among them."""
    T = 2049
    g = rng(124, E, G, k)
    s = (g.integers(0, 9, (T, E)) / 8).astype(np.float32)
    s[::2] = g.random((s[::2].shape), dtype=np.float32)
    s[5] = 0.0
    bias = (g.integers(-2, 3, E) / 8).astype(np.float32)
    bias[g.integers(0, E, E // 8)] = -np.inf
    out = []
    for n in (T, T - 1, 70, 1):
        cfg = L.make_cfg(T=n, H=64, E=E, k=k, G=G, M=M, S=0, I=128, group_topr=topr, act="bf16")
        sd = dev_f32(s[:n])
        idx = torch.full((n, k), -1, dtype=torch.int32, device="cuda")
        w = torch.full((n, k), -1.0, device="cuda")
        L.moe_route(cfg, None, None, None, dev_f32(bias), sd, L.MOE_SCORES_IN | flags, idx, w, None)
        out.append((host(idx), host(w)))
    with np.errstate(invalid="ignore"):
        for idx, w in out[1:]:
            np.testing.assert_array_equal(idx, out[0][0][:len(idx)])
            np.testing.assert_array_equal(w.view(np.uint32), out[0][1][:len(w)].view(np.uint32))


def test_a_token_that_no_expert_may_take():
    """Every logit -inf: affinities and gates of 0, the experts chosen by the bias alone."""
    for T, E, G in ((3, 16, 4), (2100, 256, 8), (5, 13, 1)):
        x, w, bias = _inputs(T, 64, E, "bf16")
        cfg = L.make_cfg(T, 64, E, G, 1, 2, 0, 128, 1, 1.0, "bf16", "bf16")
        o = dev_f32(np.full(E, -np.inf, np.float32))
        say(f"softmax, all masked T={T} E={E}")
        for flags in (L.MOE_SOFTMAX, L.MOE_SOFTMAX | L.MOE_GATES_RAW):
            s, idx, gates = _route(cfg, to_device(f32_to_bf16_bits(x)), to_device(f32_to_bf16_bits(w)), o, dev_f32(bias),
                                   flags, True)
            ir, _ = oracle.route(np.zeros((T, E), np.float32), bias, G, 1, 2, 1, 1.0)
            assert (s == 0).all() and (gates == 0).all() and (idx == ir).all()


@pytest.mark.parametrize("T,E", [(40, 16), (2100, 256), (30, 13), (17000, 256)])
def test_raw_sigmoid_gates(T, E):
    """MOE_GATES_RAW alone: the sigmoid's selection, gates scale * s; and on given affinities."""
    x, w, bias = _inputs(T, 128, E, "bf16")
    cfg = L.make_cfg(T, 128, E, 1, 1, 4, 0, 128, 1, 2.5, "bf16", "bf16")
    xd, wd = to_device(f32_to_bf16_bits(x)), to_device(f32_to_bf16_bits(w))
    say(f"raw sigmoid gates T={T} E={E}")
    s, idx, gates = _route(cfg, xd, wd, None, dev_f32(bias), L.MOE_GATES_RAW, True)
    s0, idx0, _ = _route(cfg, xd, wd, None, dev_f32(bias), 0, True)
    assert (s == s0).all() and (idx == idx0).all()
    assert (gates == np.float32(2.5) * np.take_along_axis(s, idx.astype(np.int64), 1)).all()
    sd = dev_f32(s)
    gi, gg = torch.empty((T, 4), dtype=torch.int32, device="cuda"), torch.empty((T, 4), device="cuda")
    L.moe_route(cfg, None, None, None, dev_f32(bias), sd, L.MOE_SCORES_IN | L.MOE_GATES_RAW, gi, gg)
    torch.cuda.synchronize()
    assert (host(gi) == idx).all() and (host(gg) == gates).all() and (host(sd) == s).all()


BACKWARD = [
    # (T, H, E, k, alpha, seq)
    (1, 64, 4, 1, 0.0, 0),
    (64, 128, 16, 4, 0.1, 16),
    (300, 256, 64, 6, 0.0, 0),
    (130, 192, 13, 3, 0.2, 65),
    (1100, 384, 256, 8, 0.01, 0),
    (257, 64, 300, 16, 0.0, 0),
    (2048, 128, 512, 8, 0.05, 512),
    (1200, 64, 16, 2, 0.05, 1),            # 1200 partial losses, 1024 and 1032
    (256, 64, 256, 4, 0.05, 1),
    (129, 64, 512, 4, 0.05, 1),
]


@pytest.mark.parametrize("flags", [L.MOE_SOFTMAX, L.MOE_SOFTMAX | L.MOE_GATES_RAW, L.MOE_GATES_RAW])
@pytest.mark.parametrize("T,H,E,k,alpha,seq", BACKWARD)
def test_route_backward(T, H, E, k, alpha, seq, flags):
    say(f"route backward T={T} H={H} E={E} k={k} alpha={alpha} flags={flags}")
    softmax, raw = bool(flags & L.MOE_SOFTMAX), bool(flags & L.MOE_GATES_RAW)
    x, w, bias = _inputs(T, H, E, "bf16", 1)
    s = oracle.affinity_softmax(x, w) if softmax else oracle.affinity(x, w)
    idx, _ = oracle.route(s, bias, 1, 1, k, 1, 2.5)
    dg = rng(123, T, k).standard_normal((T, k)).astype(np.float32)
    cfg = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 2.5, "bf16", "bf16")
    ws = torch.full((L.moe_workspace_bytes(cfg, L.MOE_WS_ROUTE_BWD_SOFTMAX),), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dw, loss = (torch.full(sh, float("nan"), device="cuda") for sh in ((T, H), (E, H), (1,)))
    L.moe_route_backward_flags(cfg, flags, to_device(f32_to_bf16_bits(x)), to_device(f32_to_bf16_bits(w)), dev_f32(s),
                               dev_i32(idx), dev_f32(dg), alpha, seq, dx, dw, loss, ws)
    torch.cuda.synchronize()
    dxr, dwr, lr = oracle.route_backward(x, w, s, idx, dg, 2.5, alpha, seq, softmax, raw)
    # the magnitudes that dlogit is made of
    p = s.astype(np.float64)
    sel = np.take_along_axis(p, idx.astype(np.int64), 1)
    S = sel.sum(axis=1, keepdims=True)
    a = 2.5 * np.abs(dg) if raw else 2.5 / S * (np.abs(dg) + (np.abs(dg) * sel).sum(axis=1, keepdims=True) / S)
    A = np.zeros((T, E))
    np.put_along_axis(A, idx.astype(np.int64), a, axis=1)
    if alpha:
        Lq = seq or T
        f = E / k                                                              # (f_e is at most E / k)
        A += 2 * alpha * f / T / p.sum(axis=1, keepdims=True)
    mag = p * (A + (p * A).sum(axis=1, keepdims=True)) if softmax else p * A
    dl = 100 * EPS32 * mag + 2.0 ** -17 * mag
    tol_x = dl @ np.abs(w) + (2 * E + 8) * EPS32 * (mag @ np.abs(w))
    tol_w = dl.T @ np.abs(x) + (2 * T + 8) * EPS32 * (mag.T @ np.abs(x))
    assert (np.abs(host(dx) - dxr) <= tol_x).all()
    assert (np.abs(host(dw) - dwr) <= tol_w).all()
    assert abs(host(loss)[0] - lr) <= (T + E + 40) * EPS32 * abs(lr)
    keep = host(dw).copy()
    dw.fill_(float("nan"))                                                     # without dx: the same dw
    L.moe_route_backward_flags(cfg, flags, to_device(f32_to_bf16_bits(x)), to_device(f32_to_bf16_bits(w)), dev_f32(s),
                               dev_i32(idx), dev_f32(dg), alpha, seq, None, dw, loss, ws)
    torch.cuda.synchronize()
    assert (host(dw) == keep).all()


def test_route_backward_of_a_masked_token():
    """A token without any affinity gives no gradient and no NaN; an id outside the experts is passed over."""
    T, H, E, k = 6, 64, 8, 2
    x, w, _ = _inputs(T, H, E, "bf16", 2)
    s = oracle.affinity_softmax(x, w)
    s[2] = 0
    idx = np.tile(np.array([[1, 3]], np.int32), (T, 1))
    idx[4, 1], idx[5, 0] = 8, -1
    cfg = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 1.0, "bf16", "bf16")
    ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_ROUTE_BWD_SOFTMAX), dtype=torch.uint8, device="cuda")
    for flags in (L.MOE_SOFTMAX, L.MOE_SOFTMAX | L.MOE_GATES_RAW):
        dx, dw, loss = (torch.full(sh, float("nan"), device="cuda") for sh in ((T, H), (E, H), (1,)))
        say(f"route backward, masked token, flags={flags}")
        L.moe_route_backward_flags(cfg, flags, to_device(f32_to_bf16_bits(x)), to_device(f32_to_bf16_bits(w)), dev_f32(s),
                                   dev_i32(idx), dev_f32(np.ones((T, k))), 0.0, 0, dx, dw, loss, ws)
        torch.cuda.synchronize()
        assert (host(dx)[2] == 0).all() and np.isfinite(host(dx)).all() and np.isfinite(host(dw)).all()
