"""Training steps of shares and of padded batches, beyond the single calls."""
import numpy as np
import pytest
import torch

from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import MoeLayerGPU, to_device
from gpu_util import dev_f32, dev_i32, host, rel_inf, say
from oracle.backward import backward_from_routing
from oracle.layer import decode_act
from workloads import MID
from workloads.inputs import f32_to_bf16_bits, make_weights, make_x, rng

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8       # half a step of bf16, relative


def _dy(c, seed):
    return f32_to_bf16_bits(rng(seed, c.T).standard_normal((c.T, c.H)).astype(np.float32))


def test_shares_with_the_balance_loss():
    """Two shares, the first of which adds the balance loss: dx, the router's gradient and the loss sum to the whole
    layer's.  Every dx and dlogit is rounded to bf16 on its own, the whole layer's and each share's.  In half steps of
    the largest value, with the oracle's dlogit on these inputs and every sign against us: dx 3 for its own roundings
    and 2 through dlogit, the router's gradient 8.3; the rest of the 8 and 12 that are allowed is for the gates'
    gradients, whose rows of y are rounded in either layer.  A balance term counted twice is 160 and 250."""
    c = MID.with_(T=260, H=256, E=16, G=4, M=2, k=4, S=1, I=256)
    wts, alpha = make_weights(c), 2000.0
    x, dy, bias = to_device(make_x(c)), to_device(_dy(c, 91)), dev_f32(wts.bias0)
    say("balance loss of shares")

    def step(layer, a):
        layer.forward(x, bias)
        dx = host(layer.backward(x, dy, a, 65)).astype(np.float64)
        torch.cuda.synchronize()
        return dx, host(layer.g_w_router).astype(np.float64), float(host(layer.loss_bal)[0])

    whole = MoeLayerGPU(c, wts)
    dx0, gr0, _ = step(whole, 0.0)
    dx, gr, loss = step(whole, alpha)
    first = step(MoeLayerGPU(c, wts, share=(0, 7), adds_balance=True), alpha)
    rest = step(MoeLayerGPU(c.with_(S=0), wts, share=(7, 9)), 0.0)
    assert first[2] == loss > 0 and rest[2] == 0
    for steps, one, two, want, without in ((8, first[0], rest[0], dx, dx0), (12, first[1], rest[1], gr, gr0)):
        tol = steps * BF * np.abs(want).max()
        assert np.abs(want - without).max() > 10 * tol
        assert np.abs(one + two - want).max() <= tol


GRADS = ("dx", "d_topk_w", "g_w_gate_up", "g_w_down", "g_ws_gate_up", "g_ws_down", "g_w_router")
PADDED = {
    "recomputed": (MID.with_(T=260, H=256, E=16, G=4, M=2, k=4, S=2, I=256), 133, {}),
    "saved": (MID.with_(T=260, H=256, E=16, G=4, M=2, k=4, S=1, I=256), 133, dict(save_gu=True)),
    "no shared experts": (MID.with_(T=100, H=320, E=10, G=2, M=1, k=3, S=0, I=128), 37, {}),
    "share": (MID.with_(T=260, H=256, E=16, G=4, M=2, k=4, S=1, I=256), 133, dict(share=(5, 8))),
    "none live": (MID.with_(T=70, H=256, E=16, G=4, M=2, k=4, S=1, I=128), 0, {}),
    "all live": (MID.with_(T=70, H=256, E=16, G=4, M=2, k=4, S=1, I=128), 70, {}),
}


def _gradients(layer):
    return {n: getattr(layer, n).clone() for n in GRADS if getattr(layer, n) is not None}


def _same(a, b, what):
    for n in a:
        assert torch.equal(a[n].view(torch.int8), b[n].view(torch.int8)), f"{what}: {n}"


@pytest.mark.parametrize("name", PADDED)
def test_padded_training_step(name):
    """What lies in the padded rows of x and dy reaches no gradient: NaN, infinities and numbers there give the bits
    that zeros give, and the gradients are the live tokens' (against the oracle on those alone, normwise with the
    2e-2 that bf16 operands are allowed in a whole batch's backward pass)."""
    c, live, kw = PADDED[name]
    wts = make_weights(c)
    x, dy, bias = to_device(make_x(c)), to_device(_dy(c, 92)), dev_f32(wts.bias0)
    n = torch.tensor([live], dtype=torch.int32, device="cuda")
    layer = MoeLayerGPU(c, wts, **kw)
    layer.alloc_backward()
    say(f"padded training step, {name}")

    def step(fill_x, fill_dy):
        xs, ds = x.clone(), dy.clone()
        xs[live:], ds[live:] = fill_x, fill_dy
        before = xs.clone(), ds.clone()
        layer.forward(xs, bias, n_tokens=n)
        layer.backward(xs, ds)
        torch.cuda.synchronize()
        for now, then in zip((xs, ds), before):      # the caller's own
            assert torch.equal(now.view(torch.int16), then.view(torch.int16))
        return _gradients(layer)

    clean = step(0.0, 0.0)
    for fill_x, fill_dy in ((1.0, 1000.0), (float("nan"), 0.0), (0.5, float("nan")), (float("inf"), float("-inf"))):
        _same(clean, step(fill_x, fill_dy), f"padded rows of x {fill_x}, of dy {fill_dy}")
    for n_ in ("dx", "d_topk_w"):
        assert not clean[n_][live:].any(), n_
    if "share" in kw or live == 0:
        if live == 0:
            assert not any(v.any() for v in clean.values())
        return
    f64 = lambda a: decode_act(a).astype(np.float64)
    idx = host(layer.topk_idx)[:live].astype(np.int64)
    o = backward_from_routing(f64(make_x(c))[:live], f64(wts.w_router), wts.logit_offset, f64(wts.w_gate_up),
                              f64(wts.w_down), [f64(a) for a in wts.ws_gate_up] if c.S else None,
                              [f64(a) for a in wts.ws_down] if c.S else None, idx, f64(_dy(c, 92))[:live],
                              c.route_scale)
    got = {k: host(v) for k, v in clean.items()}
    errs = {"dx": rel_inf(got["dx"][:live], o["dx"]), "d_topk_w": rel_inf(got["d_topk_w"][:live], o["dw"]),
            "dw_router": rel_inf(got["g_w_router"], o["dw_router"])}
    for e in range(c.E):
        if (idx == e).any():
            errs[f"dw_gate_up[{e}]"] = rel_inf(got["g_w_gate_up"][e], o["dw_gate_up"][e])
            errs[f"dw_down[{e}]"] = rel_inf(got["g_w_down"][e], o["dw_down"][e])
        else:
            assert not got["g_w_gate_up"][e].any() and not got["g_w_down"][e].any()
    if c.S:
        errs["dws_gate_up"] = rel_inf(got["g_ws_gate_up"], o["dws_gate_up"])
        errs["dws_down"] = rel_inf(got["g_ws_down"], o["dws_down"])
    bad = {k: v for k, v in errs.items() if not v < 2e-2}
    assert not bad, bad


@pytest.mark.parametrize("save_gu", [False, True])
def test_padded_training_step_replays(save_gu):
    """Forward and backward of a padded batch in one graph follow the live count from replay to replay, with an eager
    step's bits, whatever the padded rows hold."""
    c = MID.with_(T=200, H=256, E=16, G=4, M=2, k=4, S=1, I=256)
    wts = make_weights(c)
    bias = dev_f32(wts.bias0)
    eager, graph = MoeLayerGPU(c, wts, save_gu=save_gu), MoeLayerGPU(c, wts, save_gu=save_gu)
    xg, dg = to_device(make_x(c)), to_device(_dy(c, 93))
    ng = torch.tensor([c.T], dtype=torch.int32, device="cuda")
    say(f"padded training step in a graph, save_gu={save_gu}")
    graph.alloc_backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.forward(xg, bias, n_tokens=ng)
        graph.backward(xg, dg)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.forward(xg, bias, n_tokens=ng)
        graph.backward(xg, dg)
    for step, live in enumerate((200, 1, 0, 133, 200)):
        xs, ds = to_device(make_x(c, step)), to_device(_dy(c, 94 + step))
        xs[live:] = float("nan") if step % 2 else 1.0
        ds[live:] = float("nan") if step % 2 == 0 else 1.0
        xg.copy_(xs)
        dg.copy_(ds)
        ng.fill_(live)
        eager.forward(xs, bias, n_tokens=torch.tensor([live], dtype=torch.int32, device="cuda"))
        eager.backward(xs, ds)
        want = _gradients(eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _same(want, _gradients(graph), f"replay {step}")
        assert all(torch.isfinite(v).all() for v in want.values()), step


@pytest.mark.parametrize("E,k", [(16, 4), (70, 3), (512, 8)])
def test_router_gradient_passes_over_foreign_ids(E, k):
    """Ids outside [0, E) where no gate gradient comes from: the router's gradients have the bits that real ids give
    there, and the loss counts the others (fp32 sums over a sequence: 1e-4, as for whole batches)."""
    T, H, L_, alpha, scale = 96, 128, 32, 0.5, 2.5
    g = rng(95, E, k)
    cfg = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, scale, "bf16", "bf16")
    bits = lambda *s: to_device(f32_to_bf16_bits(g.standard_normal(s).astype(np.float32)))
    x, w = bits(T, H), bits(E, H)
    s = g.uniform(0.05, 0.95, (T, E)).astype(np.float32)
    idx = np.argsort(g.random((T, E)), axis=1)[:, :k].astype(np.int32)
    dead = g.random(T) < 0.4
    dw = g.standard_normal((T, k)).astype(np.float32)
    dw[dead] = 0
    foreign = idx.copy()
    foreign[dead] = g.choice(np.array([-1, E, 511 + 1, -2 ** 31, 2 ** 31 - 1], np.int32), (dead.sum(), k))
    say(f"foreign ids E={E} k={k}")

    def run(ids, a):
        out = (torch.empty((T, H), dtype=torch.float32, device="cuda"),
               torch.empty((E, H), dtype=torch.float32, device="cuda"), torch.empty(1, device="cuda"))
        ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_ROUTE_BWD), dtype=torch.uint8, device="cuda")
        L.moe_route_backward(cfg, x, w, dev_f32(s), dev_i32(ids), dev_f32(dw), a, L_, *out, ws)
        torch.cuda.synchronize()
        return out

    for got, want in zip(run(foreign, 0.0), run(idx, 0.0)):
        assert torch.equal(got, want)
    P = s.astype(np.float64) / s.sum(1, dtype=np.float64, keepdims=True)
    loss = 0.0
    for b in range(T // L_):
        rows = slice(b * L_, (b + 1) * L_)
        count = np.bincount(idx[rows][~dead[rows]].reshape(-1), minlength=E)
        loss += alpha / (T // L_) * (E / (k * L_) * count * P[rows].mean(0)).sum()
    dx, dr, got = run(foreign, alpha)
    assert torch.isfinite(dx).all() and torch.isfinite(dr).all()
    assert abs(float(got) - loss) <= 1e-4 * loss
