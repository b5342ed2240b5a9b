"""GPU parity of the routing and its gradients where a token has no affinity at all (every logit -inf), and of empty
batches.

Bounds (fixed before the first run).  The loss: (T + E + 40) 2^-24 of itself, as for batches without such tokens.
Gradients: dlogit is off by 100 2^-24 of the magnitudes that make it up, and by half a step of what it is stored as: one
bf16 number (2^-8, moe_route_backward) or two (2^-17, with flags).  A product over n terms adds (2 n + 8) 2^-24 of the sum
of magnitudes."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import to_device
from gpu_util import dev_f32, host, say
from route_grad_util import EPS32, backward, bounds, grid
from workloads.inputs import f32_to_bf16_bits, rng

pytestmark = pytest.mark.gpu

FLAGS = [None, L.MOE_SOFTMAX, L.MOE_SOFTMAX | L.MOE_GATES_RAW, L.MOE_GATES_RAW]   # None: moe_route_backward


@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("T,H,E,k,alpha,seq", [(6, 64, 8, 2, 0.5, 0), (128, 64, 13, 3, 0.5, 32), (130, 128, 256, 8, 0.5, 65),
                                               (600, 64, 60, 4, 0.0, 0), (1200, 64, 16, 2, 0.3, 1), (70, 64, 300, 5, 0.5, 7)])
def test_a_token_without_affinities(T, H, E, k, alpha, seq, flags):
    say(f"route backward, tokens without affinities, T={T} E={E} alpha={alpha} flags={flags}")
    g = rng(202, T, H, E)
    x, w = grid(g, T, H, 1.0, 2.0 ** -3, 32), grid(g, E, H, 1.5 / np.sqrt(H), 2.0 ** -11, 61)
    softmax, raw = bool((flags or 0) & L.MOE_SOFTMAX), bool((flags or 0) & L.MOE_GATES_RAW)
    s = oracle.affinity_softmax(x, w) if softmax else oracle.affinity(x, w)
    none = np.array([0, T // 2, T - 1])
    s[none] = 0
    idx, _ = oracle.route(s, (g.uniform(-0.1, 0.1, E) / E).astype(np.float32), 1, 1, k, 1, 2.5)
    dg = g.standard_normal((T, k)).astype(np.float32)
    cfg = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 2.5, "bf16", "bf16")
    dx, dw, loss = backward(cfg, flags, x, w, s, idx, dg, alpha, seq)
    dxr, dwr, lr = oracle.route_backward(x, w, s, idx, dg, 2.5, alpha, seq, softmax, raw)
    tx, tw = bounds(x, w, s, idx, dg, alpha, softmax, raw, 1 if flags is None else 2)
    assert np.isfinite(dx).all() and np.isfinite(dw).all() and np.isfinite(loss)
    assert (dx[none] == 0).all()
    assert abs(loss - lr) <= (T + E + 40) * EPS32 * abs(lr) and (lr > 0) == (alpha > 0)
    assert (np.abs(dx - dxr) <= tx).all() and (np.abs(dw - dwr) <= tw).all()


@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("H,E", [(64, 1), (192, 13), (4096, 512)])
def test_an_empty_batch(H, E, flags):
    """Sums over no token: a weight gradient and a loss of 0, and nothing written behind them."""
    say(f"route backward, empty batch, H={H} E={E} flags={flags}")
    cfg = L.make_cfg(0, H, E, 1, 1, 1, 0, 128, 1, 2.5, "bf16", "bf16")
    nan = lambda n: torch.full((n,), float("nan"), device="cuda")
    one = torch.zeros(16, dtype=torch.bfloat16, device="cuda")            # (there has to be some address)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    for alpha, with_dx in ((0.0, True), (0.5, False)):
        dw, loss, dx = nan(E * H + 4), nan(2), nan(4)
        kind = L.MOE_WS_ROUTE_BWD if flags is None else L.MOE_WS_ROUTE_BWD_SOFTMAX
        ws = torch.full((L.moe_workspace_bytes(cfg, kind),), 0xFF, dtype=torch.uint8, device="cuda")
        args = (one, one, nan(4), ids, nan(4), alpha, 0, dx if with_dx else None, dw, loss, ws)
        if flags is None:
            L.moe_route_backward(cfg, *args)
        else:
            L.moe_route_backward_flags(cfg, flags, *args)
        torch.cuda.synchronize()
        dw, loss = host(dw), host(loss)
        assert (dw[:E * H] == 0).all() and np.isnan(dw[E * H:]).all()
        assert loss[0] == 0 and np.isnan(loss[1]) and np.isnan(host(dx)).all()


@pytest.mark.parametrize("S", [0, 2])
@pytest.mark.parametrize("saved", [False, True])
def test_the_experts_gradients_of_an_empty_batch(S, saved):
    say(f"expert gradients, empty batch, S={S} saved={saved}")
    E, H, I = 3, 192, 128
    cfg = L.make_cfg(0, H, E, 1, 1, 1, S, I, 1, 1.0, "bf16", "bf16")
    nan = lambda n: torch.full((n + 4,), float("nan"), device="cuda")
    sizes = [E * 2 * I * H, E * H * I] + ([S * 2 * I * H, S * H * I] if S else [])
    out = [nan(n) for n in sizes]
    grads = L.expert_grads(*(out if S else out + [None, None]))
    one = torch.zeros(64, dtype=torch.bfloat16, device="cuda")            # (there has to be some address)
    sh = (one, one) if S else (None, None)
    w = L.expert_weights(one, one, *sh)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    ws = torch.full((L.moe_workspace_bytes(cfg, L.MOE_WS_FFN_BWD),), 0xFF, dtype=torch.uint8, device="cuda")
    if saved:
        keep = L.ffn_saved(one, one, *sh)
        L.moe_expert_ffn_backward_saved(cfg, one, one, offsets, w, keep, one, one, one, one, grads, ws)
    else:
        L.moe_expert_ffn_backward(cfg, one, one, offsets, w, one, one, one, one, grads, ws)
    torch.cuda.synchronize()
    for t, n in zip(out, sizes):
        g = host(t)
        assert (g[:n] == 0).all() and np.isnan(g[n:]).all()
    assert (host(one) == 0).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,G,k", [(9, 256, 8, 8), (2100, 256, 8, 8), (17000, 256, 8, 8), (9, 64, 4, 6), (5000, 16, 4, 4),
                                     (9, 60, 5, 20), (70, 300, 3, 32)])
def test_gates_of_a_token_without_affinities(T, E, G, k, act):
    """Gates of 0 on every path: affinities given (a softmax's own with masked tokens among them), a sigmoid of masked
    logits, and a softmax.  The other tokens' gates are what they are without such tokens, bit for bit."""
    if act == "f32" and T > 3000:
        return
    say(f"gates without affinities T={T} E={E} {act}")
    g = rng(203, T, E)
    s = g.random((T, E)).astype(np.float32)
    none = np.array([1, T - 1])
    bias = (g.uniform(-0.1, 0.1, E)).astype(np.float32)
    cfg = L.make_cfg(T, 64, E, G, G, k, 0, 128, 1, 2.5, act, act)
    run = lambda flags, x, w, o, sc: _route(cfg, flags, x, w, o, bias, sc)
    want_i, want_g = run(L.MOE_SCORES_IN, None, None, None, s)
    masked = s.copy()
    masked[none] = 0
    idx, gates = run(L.MOE_SCORES_IN, None, None, None, masked)
    rest = np.delete(np.arange(T), none)
    ir, _ = oracle.route(masked, bias, G, G, k, 1, 2.5)
    assert (idx == ir).all() and (gates[none] == 0).all()
    assert (gates[rest] == want_g[rest]).all() and (idx[rest] == want_i[rest]).all()
    up = dev_f32 if act == "f32" else (lambda a: to_device(f32_to_bf16_bits(a)))
    x, w = up(grid(g, T, 64, 1.0, 2.0 ** -3, 32)), up(grid(g, E, 64, 0.2, 2.0 ** -11, 61))
    o = dev_f32(np.full(E, -np.inf))
    for flags in (0, L.MOE_SOFTMAX):
        idx, gates = run(flags, x, w, o, None)
        ir, _ = oracle.route(np.zeros((1, E), np.float32), bias, G, G, k, 1, 2.5)
        assert (gates == 0).all() and (idx == ir).all()


def _route(cfg, flags, x, w, o, bias, s):
    idx = torch.full((cfg.T, cfg.k), -1, dtype=torch.int32, device="cuda")
    gates = torch.full((cfg.T, cfg.k), float("nan"), device="cuda")
    ws = torch.empty(L.moe_workspace_bytes(cfg, L.MOE_WS_ROUTE), dtype=torch.uint8, device="cuda")
    L.moe_route(cfg, x, w, o, dev_f32(bias), None if s is None else dev_f32(s), flags, idx, gates, ws)
    torch.cuda.synchronize()
    return host(idx), host(gates)


@pytest.mark.parametrize("small", [2.0 ** -126, 1e-40, 2.0 ** -146])
@pytest.mark.parametrize("T,E,k,alpha,flags", [(8, 16, 1, 0.0, L.MOE_SOFTMAX), (70, 64, 4, 0.0, L.MOE_SOFTMAX),
                                               (70, 256, 8, 0.2, L.MOE_SOFTMAX), (40, 100, 3, 0.2, L.MOE_GATES_RAW),
                                               (8, 16, 1, 0.0, None), (70, 64, 4, 0.0, None), (70, 256, 8, 0.2, None)])
def test_gradients_of_vanishing_affinities(T, E, k, alpha, flags, small):
    """Tokens whose selected affinities (a softmax under a bias that forces them), or all of them (a sigmoid), are next to
    nothing: gates and normalised affinities are their ratios, and the gradient has the size of those."""
    say(f"route backward, affinities of {small}, T={T} E={E} k={k} flags={flags}")
    g = rng(204, T, E, k)
    softmax, raw, H = flags == L.MOE_SOFTMAX, flags == L.MOE_GATES_RAW, 64
    x, w = grid(g, T, H, 1.0, 2.0 ** -3, 32), grid(g, E, H, 0.2, 2.0 ** -11, 61)
    s = (small * g.integers(1, 9, (T, E))).astype(np.float32)
    if softmax:
        s[:, E - 1] = 1
    idx = np.stack([g.permutation(E - 1)[:k] for _ in range(T)]).astype(np.int32)
    dg = g.standard_normal((T, k)).astype(np.float32)
    cfg = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 2.5, "bf16", "bf16")
    dx, dw, loss = backward(cfg, flags, x, w, s, idx, dg, alpha, 0)
    dxr, dwr, lr = oracle.route_backward(x, w, s, idx, dg, 2.5, alpha, 0, softmax, raw)
    tx, tw = bounds(x, w, s, idx, dg, alpha, softmax, raw, 1 if flags is None else 2)
    assert (np.abs(dx - dxr) <= tx).all() and (np.abs(dw - dwr) <= tw).all()
    # (a rounding below 2^-126 is off by half a step of 2^-149, not by 2^-24 of the number: E sums of T + 40 shares, each
    # times f <= E / k and alpha / T.  It counts where the loss itself has vanished.)
    under = (T + E + 40) * 2.0 ** -150 * E * (E / k)
    assert abs(loss - lr) <= (T + E + 40) * EPS32 * abs(lr) + under
    assert np.abs(dxr).max() > (1e-6 if k > 1 else -1)    # (no vanishing gradient; with one expert its gate is a constant)
