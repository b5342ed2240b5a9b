"""GPU parity of moe_norm and moe_norm_backward with the formulas in 64 bits.

Bounds (fixed before the first run).  A row's sums of n terms are chains of at most 128 + H / 512 additions on a lane
and a tree: C 2^-24 of the sum of magnitudes, C = 150 + H / 256 with the handful of roundings around them.  h w is
exact for bf16 (a product of two 8-bit significands), r is off by C 2^-24 at most, and a bf16 result by another 2^-8 of
its value (half a step), an fp32 one by 2^-24.  int8 codes and E4M3 codes are functions of h w alone and are compared
bit for bit; their scales like r.  dweight adds T terms: T + C times 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import to_device
from gpu_util import host, say
from workloads.inputs import f32_to_bf16_bits, rng

pytestmark = pytest.mark.gpu

EPS32, BF = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6


def _cfg(T, H, act, wgt):
    return L.make_cfg(T, H, 1, 1, 1, 1, 0, 128, 1, 1.0, act, wgt)


def _rows(T, H, act, *salt):
    """Stored values (bf16 bits or fp32) with outlying channels and row magnitudes over some binades."""
    g = rng(111, T, H, *salt)
    v = g.standard_normal((T, H)) * (1 + 20 * (g.random(H) > 0.99)) * np.exp2(g.integers(-6, 6, (T, 1)))
    v = v.astype(np.float32)
    return v if act == "f32" else f32_to_bf16_bits(v)


def _weight(H, act):
    w = (1 + 0.2 * rng(112, H).standard_normal(H)).astype(np.float32)
    return w if act == "f32" else f32_to_bf16_bits(w)


def _fill(shape, dtype):
    return torch.full(shape, 3, dtype=dtype, device="cuda")


FORWARD = [
    # (T, H, act, codes, residual, y, live)
    (1, 7168, "bf16", "int8", True, True, None),
    (1, 128, "bf16", "int8", False, True, None),
    (5, 384, "bf16", "fp8_e4m3", True, False, None),
    (7, 8192, "bf16", "fp8_e4m3", False, True, 5),
    (3, 8320, "bf16", "int8", True, True, None),        # longer than the registers of a wavefront's row hold
    (3, 17024, "bf16", "int8", True, True, 2),          # ... and of a workgroup's: read again from h
    (2, 33408, "bf16", "int8", False, False, None),
    (3, 17408, "bf16", None, True, True, None),
    (300, 192, "bf16", None, True, True, 0),
    (2100, 128, "bf16", "int8", True, True, 2001),      # a wavefront a row
    (2049, 1408, "bf16", "fp8_e4m3", True, True, 1),
    (2050, 7168, "bf16", "int8", False, False, None),
    (2300, 64, "bf16", None, False, True, None),
    (1, 4, "f32", None, True, True, None),
    (77, 132, "f32", None, True, True, 70),
    (2100, 1000, "f32", None, False, True, None),
    (4, 20004, "f32", None, True, True, 3),
    (70, 2048, "bf16", "int8", True, True, None),       # one and two wavefronts a row, exactly and hardly filled
    (9, 4096, "bf16", "int8", True, True, None),
    (2300, 2176, "bf16", "fp8_e4m3", True, True, 2299),
    (50, 2048, "f32", None, True, True, None),
]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("T,H,act,codes,residual,with_y,live", FORWARD)
def test_norm(T, H, act, codes, residual, with_y, live, inplace):
    say(f"norm T={T} H={H} {act} {codes} residual={residual} live={live} inplace={inplace}")
    dt = torch.float32 if act == "f32" else torch.bfloat16
    xb, wb = _rows(T, H, act, 0), _weight(H, act)
    rb = _rows(T, H, act, 1) if residual else None
    x, res, w = to_device(xb), to_device(rb), to_device(wb)
    h = (res if residual else x) if inplace else _fill((T, H), dt)
    before = host(h).copy()
    y = _fill((T, H), dt) if with_y else None
    q = s = None
    if codes:
        q = _fill((T, H), torch.int8)
        s = _fill((T,) if codes == "int8" else (T, H // 128), torch.float32)
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    L.moe_norm(_cfg(T, H, act, codes or act), n, x, res, w, EPS, h, y, q, s)
    torch.cuda.synchronize()
    m = T if live is None else live
    want = oracle.decode_act(xb)
    if residual:
        want = want + oracle.decode_act(rb)                                    # one fp32 addition
        want = want if act == "f32" else oracle.decode_act(f32_to_bf16_bits(want))
    assert (host(h)[:m] == want[:m]).all() and (host(h)[m:] == before[m:]).all()
    w64 = oracle.decode_act(wb).astype(np.float64)
    yr, r = oracle.rms_norm(want[:m], w64, EPS)
    C = (150 + H / 256) * EPS32
    if with_y:
        assert (np.abs(host(y)[:m] - yr) <= np.abs(yr) * ((EPS32 if act == "f32" else BF) + 1.01 * C)).all()
        assert (host(y)[m:] == 3).all()
    if codes:
        p = want[:m].astype(np.float64) * w64
        if codes == "int8":
            qr, sr = oracle.quantize_int8(p) if m else (np.zeros((0, H)), np.zeros(0))
            got = host(q)[:m]
        else:
            qr, sr = oracle.quantize_rows_1x128(p.astype(np.float32))
            got = host(q)[:m].view(np.uint8)
            r = r[:, None]
        assert (got == qr).all() and (host(q)[m:] == 3).all()
        assert (np.abs(host(s)[:m] - sr * r) <= sr * r * 1.01 * C).all() and (host(s)[m:] == 3).all()


def test_norm_again_gives_the_same_bits():
    """The norm of the stored sum, without a residual, is the norm that was given with it."""
    T, H = 37, 2048
    cfg = _cfg(T, H, "bf16", "int8")
    new = lambda: (_fill((T, H), torch.bfloat16), _fill((T, H), torch.int8), _fill((T,), torch.float32))
    w, h = to_device(_weight(H, "bf16")), _fill((T, H), torch.bfloat16)
    a, b = new(), new()
    say("norm again")
    L.moe_norm(cfg, None, to_device(_rows(T, H, "bf16", 0)), to_device(_rows(T, H, "bf16", 1)), w, EPS, h, *a)
    L.moe_norm(cfg, None, h, None, w, EPS, None, *b)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T", [9, 2100])
@pytest.mark.parametrize("codes", ["int8", "fp8_e4m3"])
def test_special_rows(T, codes):
    """Rows of zeros, with a NaN, with an infinity: they reach no other row."""
    H = 256
    xb = _rows(T, H, "bf16", 2)
    xb[1], xb[2, 17], xb[3, 200] = 0, 0x7FC0, 0xFF80
    wb = _weight(H, "bf16")
    y, q = _fill((T, H), torch.bfloat16), _fill((T, H), torch.int8)
    s = _fill((T,) if codes == "int8" else (T, 2), torch.float32)
    say(f"norm special rows {codes}")
    L.moe_norm(_cfg(T, H, "bf16", codes), None, to_device(xb), None, to_device(wb), EPS, None, y, q, s)
    torch.cuda.synchronize()
    y, q, s = host(y), host(q), host(s)
    assert (y[1] == 0).all() and (q[1] == 0).all() and np.isfinite(s[1]).all()
    assert np.isnan(y[2]).all()
    rest = np.delete(np.arange(T), [1, 2, 3])
    yr, _ = oracle.rms_norm(oracle.decode_act(xb)[rest], oracle.decode_act(wb), EPS)
    assert (np.abs(y[rest] - yr) <= np.abs(yr) * (BF + 2.0 ** -16)).all() and np.isfinite(s[rest]).all()
    if codes == "int8":
        assert np.isnan(s[2:4]).all() and (q[2:4] == 0).all()


BACKWARD = [
    # (T, H, act, dh, live)
    (1, 128, "bf16", False, None),
    (1, 7168, "bf16", True, None),
    (6, 384, "bf16", True, 4),
    (300, 1408, "bf16", False, None),
    (1100, 256, "bf16", True, 1001),
    (700, 8192, "bf16", True, None),
    (5, 8320, "bf16", True, None),                       # panels
    (600, 8448, "bf16", False, 590),
    (40, 64, "bf16", False, 0),
    (1, 4, "f32", False, None),
    (256, 128, "f32", True, 201),
    (530, 4096, "f32", True, None),
    (9, 9000, "f32", True, 8),
    (2600, 512, "bf16", True, 2499),                     # a wavefront a row
    (2051, 2048, "bf16", False, None),
    (2049, 1024, "f32", True, None),
]


@pytest.mark.parametrize("inplace", [None, "dy", "dh"])
@pytest.mark.parametrize("T,H,act,with_dh,live", BACKWARD)
def test_norm_backward(T, H, act, with_dh, live, inplace):
    if inplace == "dh" and not with_dh:
        return
    say(f"norm backward T={T} H={H} {act} dh={with_dh} live={live} inplace={inplace}")
    dt = torch.float32 if act == "f32" else torch.bfloat16
    hb, wb, dyb = _rows(T, H, act, 3), _weight(H, act), _rows(T, H, act, 4)
    dhb = _rows(T, H, act, 5) if with_dh else None
    dy, dh = to_device(dyb), to_device(dhb)
    dx = {None: _fill((T, H), dt), "dy": dy, "dh": dh}[inplace]
    dw = torch.full((H,), float("nan"), device="cuda")
    cfg = _cfg(T, H, act, act)
    ws = torch.full((L.moe_workspace_bytes(cfg, L.MOE_WS_NORM_BWD),), 0xFF, dtype=torch.uint8, device="cuda")
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    L.moe_norm_backward(cfg, n, to_device(hb), to_device(wb), EPS, dy, dh, dx, dw, ws)
    torch.cuda.synchronize()
    m = T if live is None else live
    f = lambda a: oracle.decode_act(a)[:m].astype(np.float64)
    h, d, w = f(hb), f(dyb), oracle.decode_act(wb).astype(np.float64)
    e = f(dhb) if with_dh else np.zeros_like(h)
    dxr, dwr = oracle.rms_norm_backward(h, w, EPS, d, e)
    _, r = oracle.rms_norm(h, w, EPS)
    u, g = np.abs(h * r[:, None]), np.abs(d * w)
    C = (150 + H / 256) * EPS32
    mag = r[:, None] * (g + u * (g * u).mean(axis=1, keepdims=True)) if m else np.zeros_like(h)
    tol = np.abs(dxr) * (EPS32 if act == "f32" else BF) * 1.01 + 3 * C * mag + 4 * EPS32 * np.abs(e)
    assert (np.abs(host(dx)[:m] - dxr) <= tol).all() and (host(dx)[m:] == 0).all()
    assert (np.abs(host(dw) - dwr) <= (2 * C + (m + 2) * EPS32) * (np.abs(d) * u).sum(axis=0)).all()


def test_norm_backward_repeats_its_bits():
    T, H = 1500, 2048
    cfg = _cfg(T, H, "bf16", "bf16")
    h, w, dy = (to_device(a) for a in (_rows(T, H, "bf16", 6), _weight(H, "bf16"), _rows(T, H, "bf16", 7)))
    ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_NORM_BWD), dtype=torch.uint8, device="cuda")
    out = []
    say("norm backward repeats")
    for _ in range(3):
        dx, dw = _fill((T, H), torch.bfloat16), _fill((H,), torch.float32)
        L.moe_norm_backward(cfg, None, h, w, EPS, dy, None, dx, dw, ws)
        out.append((dx, dw))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(o, out[0]))


def test_norm_graph_with_a_changing_live_count():
    """Forward and backward captured once, replayed on batches of other rows and live counts."""
    T, H = 64, 512
    cfg = _cfg(T, H, "bf16", "int8")
    bf = lambda: torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x, res, h, y, dy, dx = bf(), bf(), bf(), bf(), bf(), bf()
    q, s, dw = torch.zeros((T, H), dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros(H, device="cuda")
    w = to_device(_weight(H, "bf16"))
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_NORM_BWD), dtype=torch.uint8, device="cuda")

    def step(h, y, q, s, dx, dw):
        L.moe_norm(cfg, n, x, res, w, EPS, h, y, q, s)
        L.moe_norm_backward(cfg, n, h, w, EPS, dy, None, dx, dw, ws)

    say("norm graph")
    out = (h, y, q, s, dx, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*out)
    for i, live in enumerate((64, 1, 0, 40)):
        x.copy_(to_device(_rows(T, H, "bf16", 10 + i)))
        res.copy_(to_device(_rows(T, H, "bf16", 20 + i)))
        dy.copy_(to_device(_rows(T, H, "bf16", 30 + i)))
        n.fill_(live)
        eager = [t.clone() for t in out]
        step(*eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, eager)), live
