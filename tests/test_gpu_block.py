"""The norm, the routing and the experts run together, as a layer of a model runs them.

Bounds (fixed before the first run).  Outputs of a whole layer, normwise, on the routing and the 8-bit rows the GPU
made (each of those is compared on its own elsewhere): y_perm, y_shared and y are rounded to bf16 (three half steps
of 2^-8 of the largest magnitude, with every sign against us), h once more in each of its I columns, whose errors add
up like a random walk (bf16, far below a half step), so that five half steps are allowed; an E4M3 h may round to the
other neighbour where the fp32 sums differ, 2^-3 of a value in a few of its columns: two half steps more.  Gradients,
normwise: 2e-2, what bf16 operands are allowed in a whole batch's backward pass."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU, to_device
from gpu_util import dev_f32, host, rel_inf, say
from oracle.int8 import expert_int8, shared_int8
from oracle.layer import _Fp8Expert, decode_act
from workloads import MID
from workloads.inputs import f32_to_bf16_bits, make_weights, make_x, rng

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8
EPS = 1e-5


def _bits(seed, *shape):
    return f32_to_bf16_bits(rng(seed, *shape).standard_normal(shape).astype(np.float32))


def _norm_weight(c):
    return f32_to_bf16_bits((1 + 0.2 * rng(131, c.H).standard_normal(c.H)).astype(np.float32))


def _run(c, wts, layer, x, res, live):
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    y = layer.forward(to_device(x), dev_f32(wts.bias0), n_tokens=n, residual=to_device(res))
    torch.cuda.synchronize()
    return host(y)


BLOCK = {
    "int8 prefill": (MID.with_(T=600, H=512, E=16, G=4, M=2, k=4, S=2, I=384, wgt="int8"), dict(softmax=True), None),
    "int8 decode": (MID.with_(T=5, H=1408, E=32, G=8, M=3, k=6, S=1, I=128, wgt="int8"),
                    dict(softmax=True, raw_gates=True), None),
    "int8 padded": (MID.with_(T=300, H=256, E=8, G=2, M=1, k=2, S=1, I=256, wgt="int8"), dict(raw_gates=True), 171),
    "int8 no shared": (MID.with_(T=77, H=256, E=128, G=4, M=2, k=8, S=0, I=128, wgt="int8"), dict(softmax=True), None),
    "int8 one token": (MID.with_(T=1, H=512, E=16, G=4, M=2, k=4, S=1, I=128, wgt="int8"), dict(), None),
    "fp8": (MID.with_(T=300, H=512, E=16, G=4, M=2, k=4, S=1, I=256, wgt="fp8_e4m3"), dict(softmax=True), None),
    "bf16": (MID.with_(T=300, H=512, E=16, G=4, M=2, k=4, S=1, I=256), dict(softmax=True, raw_gates=True), 251),
}


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("name", BLOCK)
def test_block(name, gather):
    c, kw, live = BLOCK[name]
    wts, nw = make_weights(c), _norm_weight(c)
    x, res = make_x(c), _bits(132, c.T, c.H)
    layer = MoeLayerGPU(c, wts, gather=gather, norm=nw, eps=EPS, **kw)
    say(f"block {name} gather={gather}")
    y = _run(c, wts, layer, x, res, live)
    m = c.T if live is None else live
    h = decode_act(f32_to_bf16_bits(decode_act(x) + decode_act(res)))
    assert (host(layer.h)[:m] == h[:m]).all()
    xn = host(layer.xn)[:m].astype(np.float64)
    want, _ = oracle.rms_norm(h[:m], decode_act(nw), EPS)
    assert (np.abs(xn - want) <= np.abs(want) * (BF + 2.0 ** -16)).all()
    # the routing of the normed rows (affinities as the GPU formed them: off by the router's fp32 sums)
    s = host(layer.scores)[:m]
    aff = oracle.affinity_softmax if kw.get("softmax") else oracle.affinity
    sw = aff(xn.astype(np.float32), decode_act(wts.w_router), wts.logit_offset)
    assert (np.abs(s - sw) <= 2 * c.H * 2.0 ** -24 * np.abs(sw)
            * (1 + (np.abs(xn) @ np.abs(decode_act(wts.w_router).T.astype(np.float64))).max())).all()
    idx, gates = oracle.route(s, wts.bias0, c.G, c.M, c.k, c.group_topr, c.route_scale, raw=kw.get("raw_gates", False))
    assert (host(layer.topk_idx)[:m] == idx).all()
    assert (np.abs(host(layer.topk_w)[:m] - gates) <= 40 * 2.0 ** -24 * gates).all()
    # the experts, on the norm's codes or on the rows it wrote
    if c.wgt == "int8":
        q, qs = ((host(layer.codes)[:m], host(layer.code_scale)[:m].astype(np.float64)) if gather
                 else oracle.quantize_int8(xn))
        expert = lambda e, t: expert_int8(q[t], qs[t], decode_act(wts.w_gate_up[e]), decode_act(wts.w_down[e]))
        shared = lambda: shared_int8(q, qs, decode_act(wts.ws_gate_up), decode_act(wts.ws_down))
    elif c.wgt == "fp8_e4m3":
        q, qs = (host(layer.codes)[:m], host(layer.code_scale)[:m]) if gather else oracle.quantize_rows_1x128(
            xn.astype(np.float32))
        expert = lambda e, t: _Fp8Expert(wts.w_gate_up[e], wts.w_down[e])(q[t], qs[t])
        shared = lambda: sum(_Fp8Expert(a, b)(q, qs) for a, b in zip(wts.ws_gate_up, wts.ws_down))
    else:
        ffn = lambda r, a, b: oracle.swiglu(r, decode_act(a), decode_act(b))
        expert = lambda e, t: ffn(xn[t], wts.w_gate_up[e], wts.w_down[e])
        shared = lambda: sum(ffn(xn, a, b) for a, b in zip(wts.ws_gate_up, wts.ws_down))
    ref = shared() if c.S else np.zeros((m, c.H))
    for e in range(c.E):
        t, j = np.nonzero(idx == e)
        if len(t):
            ref[t] += expert(e, t) * gates[t, j][:, None]
    assert rel_inf(y[:m], ref) <= (7 if c.wgt == "fp8_e4m3" else 5) * BF


@pytest.mark.parametrize("wgt,gather", [("int8", True), ("int8", False), ("fp8_e4m3", True), ("bf16", True)])
def test_block_graph(wgt, gather):
    """A captured block, replayed on new rows, residuals and live counts with eager work between the replays, gives
    the eager block's bits."""
    c = MID.with_(T=310, H=512, E=16, G=4, M=2, k=4, S=1, I=256, wgt=wgt)
    wts, nw = make_weights(c), _norm_weight(c)
    kw = dict(gather=gather, norm=nw, eps=EPS, softmax=True, raw_gates=True, keep_scores=False)
    eager, graph = MoeLayerGPU(c, wts, **kw), MoeLayerGPU(c, wts, **kw)
    bias = dev_f32(wts.bias0)
    x, res = to_device(make_x(c)), to_device(_bits(133, c.T, c.H))
    n = torch.tensor([c.T], dtype=torch.int32, device="cuda")
    say(f"block graph {wgt} gather={gather}")
    graph.capture(x, bias, n_tokens=n, residual=res)
    for step, live in enumerate((310, 1, 200, 0, 309)):
        x.copy_(to_device(make_x(c, step)))
        res.copy_(to_device(_bits(134 + step, c.T, c.H)))
        n.fill_(live)
        want = eager.forward(x, bias, n_tokens=n, residual=res).clone()
        torch.cuda.synchronize()
        y = graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[:live].view(torch.int16), want[:live].view(torch.int16)), (step, live)
        assert torch.equal(graph.h.view(torch.int16), eager.h.view(torch.int16))
        assert (host(graph.topk_idx)[:live] == host(eager.topk_idx)[:live]).all()


def test_two_blocks_at_once():
    """Two layers on two streams give the bits that each gives alone."""
    layers, runs = [], []
    for i, wgt in enumerate(("int8", "int8")):
        c = MID.with_(T=700 + 60 * i, H=512, E=16, G=4, M=2, k=4, S=1, I=384, wgt=wgt)
        wts = make_weights(c)
        layers.append((MoeLayerGPU(c, wts, gather=i == 0, norm=_norm_weight(c), softmax=True), to_device(make_x(c)),
                       dev_f32(wts.bias0), to_device(_bits(141 + i, c.T, c.H))))
    say("two blocks at once")
    for layer, x, bias, res in layers:
        runs.append(layer.forward(x, bias, residual=res).clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for (layer, x, bias, res), s in zip(layers, streams):
            with torch.cuda.stream(s):
                layer.forward(x, bias, residual=res)
    torch.cuda.synchronize()
    for (layer, *_), want in zip(layers, runs):
        assert torch.equal(layer.y.view(torch.int16), want.view(torch.int16))


def test_products_past_32_bits():
    """80 copies of a batch (2.3e9 values in the sorted rows and as many in their outputs) give 80 copies of its rows."""
    c = MID.with_(T=500, H=7168, E=8, G=2, M=2, k=8, S=0, I=128, wgt="int8")
    wts, nw = make_weights(c), _norm_weight(c)
    x, bias, n = to_device(make_x(c)), dev_f32(wts.bias0), 80
    say("int8 block past 32 bits")
    small = MoeLayerGPU(c, wts, norm=nw, softmax=True)
    want = small.forward(x, bias).clone()
    ids = host(small.topk_idx)
    big = MoeLayerGPU(c.with_(T=n * c.T), wts, norm=nw, softmax=True)
    y = big.forward(x.repeat(n, 1), bias)
    torch.cuda.synchronize()
    assert big.y_perm.numel() > 1 << 31
    # (the two batches' router GEMMs add in different orders: rows that choose alike are compared)
    same = torch.from_numpy((host(big.topk_idx).reshape(n, c.T, c.k) == ids).all((0, 2))).cuda()
    assert same.float().mean() > 0.9
    y = y.reshape(n, c.T, c.H)[:, same].float()
    want = want[same].float()
    assert ((y - want).abs() <= 3 * BF * want.abs().max()).all()
    assert (y[1:] == y[0]).all()


def test_norm_past_32_bits():
    """A batch of more than 2^31 values: its last rows as they are alone."""
    T, H = 300001, 7168
    cfg = L.make_cfg(T, H, 1, 1, 1, 1, 0, 128, 1, 1.0, "bf16", "int8")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, H), dtype=torch.bfloat16, device="cuda", generator=g)
    w = torch.rand(H, device="cuda", generator=g).to(torch.bfloat16)
    say("norm past 32 bits")
    new = lambda n: (torch.empty((n, H), dtype=torch.bfloat16, device="cuda"),
                     torch.empty((n, H), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda"))
    big, m = new(T), 3000
    L.moe_norm(cfg, None, x, None, w, EPS, None, *big)
    small = new(m)
    L.moe_norm(L.make_cfg(m, H, 1, 1, 1, 1, 0, 128, 1, 1.0, "bf16", "int8"), None, x[-m:], None, w, EPS, None, *small)
    torch.cuda.synchronize()
    assert all(torch.equal(a[-m:], b) for a, b in zip(big, small))
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_NORM_BWD), dtype=torch.uint8, device="cuda")
    L.moe_norm_backward(cfg, None, x, w, EPS, big[0], None, dx, dw, ws)
    tail = torch.empty((m, H), dtype=torch.bfloat16, device="cuda")
    L.moe_norm_backward(L.make_cfg(m, H, 1, 1, 1, 1, 0, 128, 1, 1.0, "bf16", "int8"), None, x[-m:], w, EPS, small[0], None,
                        tail, dw, ws)
    torch.cuda.synchronize()
    assert torch.equal(dx[-m:], tail)


# ---------------------------------------------------------------- training
def _plain(c, wts, nw, h, idx, dy, dh, alpha, seq, softmax, raw):
    """The block in 64 bits from the norm's input h with fixed experts idx; gradients of sum(dy y) + sum(dh h) + the
    balance loss by automatic differentiation.  Returns (y, loss, gradients)."""
    t = lambda a: torch.from_numpy(decode_act(a).astype(np.float64)).requires_grad_(True)
    h = torch.from_numpy(h.astype(np.float64)).requires_grad_(True)
    w, wr, gu, dn = t(nw), t(wts.w_router), t(wts.w_gate_up), t(wts.w_down)
    sgu, sdn = (t(wts.ws_gate_up), t(wts.ws_down)) if c.S else (None, None)
    T, E = len(h), c.E
    xn = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w
    logits = xn @ wr.T
    if wts.logit_offset is not None:
        logits = logits + torch.from_numpy(wts.logit_offset.astype(np.float64))
    s = torch.softmax(logits, 1) if softmax else torch.sigmoid(logits)
    ids = torch.from_numpy(idx.astype(np.int64))
    g = torch.gather(s, 1, ids)
    g = c.route_scale * (g if raw else g / g.sum(1, keepdim=True))

    def ffn(r, a, b):
        u = r @ a.T
        return (torch.nn.functional.silu(u[:, :c.I]) * u[:, c.I:]) @ b.T

    y = sum(ffn(xn, sgu[i], sdn[i]) for i in range(c.S)) if c.S else torch.zeros_like(xn)
    for e in range(E):
        tok, j = torch.nonzero(ids == e, as_tuple=True)
        if len(tok):
            y = y.index_add(0, tok, ffn(xn[tok], gu[e], dn[e]) * g[tok, j].unsqueeze(1))
    loss = torch.zeros((), dtype=torch.float64)
    if alpha:
        n = T // seq
        f = torch.nn.functional.one_hot(ids, E).sum(1).double().reshape(n, seq, E).sum(1) * E / (c.k * seq)
        loss = alpha / n * (f * (s / s.sum(1, keepdim=True)).reshape(n, seq, E).mean(1)).sum()
    out = (y * torch.from_numpy(dy.astype(np.float64))).sum() + loss
    if dh is not None:
        out = out + (h * torch.from_numpy(dh.astype(np.float64))).sum()
    leaves = dict(dx_in=h, g_norm=w, g_w_router=wr, g_w_gate_up=gu, g_w_down=dn, g_ws_gate_up=sgu, g_ws_down=sdn)
    leaves = {k: v for k, v in leaves.items() if v is not None}
    grads = torch.autograd.grad(out, list(leaves.values()), materialize_grads=True)
    return y.detach().numpy(), float(loss.detach()), {k: v.numpy() for k, v in zip(leaves, grads)}


TRAIN = {
    "softmax, balance loss": (dict(softmax=True), 3000.0, 65, None),
    "softmax raw, saved": (dict(softmax=True, raw_gates=True, save_gu=True), 0.0, 0, None),
    "sigmoid raw": (dict(raw_gates=True), 3000.0, 130, None),
    "sigmoid": (dict(), 0.0, 0, None),
    "softmax, padded": (dict(softmax=True, save_gu=True), 0.0, 0, 133),
    "none live": (dict(softmax=True), 0.0, 0, 0),
}


@pytest.mark.parametrize("with_dh", [True, False])
@pytest.mark.parametrize("name", TRAIN)
def test_block_training_step(name, with_dh):
    kw, alpha, seq, live = TRAIN[name]
    c = MID.with_(T=260, H=256, E=16, G=4, M=2, k=4, S=1, I=256)
    wts, nw = make_weights(c), _norm_weight(c)
    x, res, dy = make_x(c), _bits(151, c.T, c.H), _bits(152, c.T, c.H)
    dh = _bits(153, c.T, c.H) if with_dh else None
    m = c.T if live is None else live
    layer = MoeLayerGPU(c, wts, norm=nw, eps=EPS, **kw)
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda")
    names = ["dx_in", "g_norm", "g_w_router", "g_w_gate_up", "g_w_down", "g_ws_gate_up", "g_ws_down"]

    def step(fill):
        dev = [to_device(a) for a in (x, res, dy)] + [to_device(dh)]
        for a in dev:
            if a is not None and fill is not None:
                a[m:] = fill
        layer.forward(dev[0], dev_f32(wts.bias0), residual=dev[1], n_tokens=n)
        layer.backward(dev[0], dev[2], alpha, seq, dh=dev[3])
        torch.cuda.synchronize()
        return {k: getattr(layer, k).clone() for k in names}

    say(f"block training step, {name}, dh={with_dh}")
    got = step(None)
    h = decode_act(f32_to_bf16_bits(decode_act(x) + decode_act(res)))[:m]
    y, loss, want = _plain(c, wts, nw, h, host(layer.topk_idx)[:m], decode_act(dy)[:m],
                           decode_act(dh)[:m] if with_dh else None, alpha, seq, kw.get("softmax", False),
                           kw.get("raw_gates", False))
    assert m == 0 or rel_inf(host(layer.y)[:m], y) <= 2e-2
    assert abs(float(host(layer.loss_bal)[0]) - loss) <= 2.0 ** -12 * loss
    for k in names:
        g = host(got[k])
        if k == "dx_in":
            assert (g[m:] == 0).all()
            g = g[:m]
        assert (np.abs(g - want[k]) <= 2e-2 * max(np.abs(want[k]).max(initial=0), 1e-30)).all(), k
    if live is not None:                       # what lies in the padded rows reaches no gradient
        for fill in (float("nan"), float("inf"), 3.0):
            again = step(fill)
            for k in names:
                assert torch.equal(again[k].view(torch.int8), got[k].view(torch.int8)), (k, fill)


def test_shares_of_a_block():
    """Two shares behind the norm, the first with the shared experts and dh: their dx and their gradients of the norm's
    weight add up to the whole block's (each share's dx is rounded to bf16 four times, the whole's too: 8 half steps)."""
    c = MID.with_(T=260, H=256, E=16, G=4, M=2, k=4, S=1, I=256)
    wts, nw = make_weights(c), _norm_weight(c)
    x, res, dy, dh = to_device(make_x(c)), *(to_device(_bits(161 + i, c.T, c.H)) for i in range(3))
    bias = dev_f32(wts.bias0)
    say("shares of a block")

    def step(layer, dh):
        layer.forward(x, bias, residual=res)
        layer.backward(x, dy, dh=dh)
        torch.cuda.synchronize()
        return [host(a).astype(np.float64) for a in (layer.dx_in, layer.g_norm, layer.g_w_router)]

    kw = dict(norm=nw, eps=EPS, softmax=True)
    whole = step(MoeLayerGPU(c, wts, **kw), dh)
    one = step(MoeLayerGPU(c, wts, share=(0, 7), **kw), dh)
    two = step(MoeLayerGPU(c.with_(S=0), wts, share=(7, 9), **kw), None)
    for a, b, w in zip(one, two, whole):
        assert np.abs(a + b - w).max() <= 8 * BF * np.abs(w).max()


def test_captured_training_step():
    """A whole training step recorded into a graph and replayed on other rows, with eager work between the replays."""
    c = MID.with_(T=260, H=256, E=16, G=4, M=2, k=4, S=1, I=256)
    wts, nw = make_weights(c), _norm_weight(c)
    kw = dict(norm=nw, eps=EPS, softmax=True, save_gu=True)
    eager, layer = MoeLayerGPU(c, wts, **kw), MoeLayerGPU(c, wts, **kw)
    x, res, dy, dh = to_device(make_x(c)), *(to_device(_bits(171 + i, c.T, c.H)) for i in range(3))
    bias = dev_f32(wts.bias0)
    names = ["dx_in", "g_norm", "g_w_router", "g_w_gate_up", "g_w_down", "g_ws_gate_up", "g_ws_down", "loss_bal"]

    def step(m):
        m.forward(x, bias, residual=res)
        m.backward(x, dy, 1000.0, 65, dh=dh)

    say("captured training step")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(layer)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(layer)
    for i in range(4):
        x.copy_(to_device(make_x(c, i)))
        dy.copy_(to_device(_bits(181 + i, c.T, c.H)))
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(getattr(layer, n).view(torch.int8), getattr(eager, n).view(torch.int8)), (i, n)
