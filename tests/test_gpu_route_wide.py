"""GPU parity of the router's gradients at the sizes of large training steps, whose dx runs in tiles of 128 x 256 (from
1024 of them on) and whose dW_r is split by what fills the chip.

Bounds (fixed before the first run): route_grad_util.bounds; the loss (T + E + 40) 2^-24 of itself.  dx is compared on
sampled tokens, the first and last of row tiles and the whole last tile among them, dW_r as a whole."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from gpu_util import say
from route_grad_util import EPS32, backward, bounds, grid
from workloads.inputs import rng

pytestmark = pytest.mark.gpu

CASES = [
    # (T, H, E, k, alpha, seq): wide tiles with a last row tile of one token and a last column tile of 64
    (16385, 2112, 256, 8, 0.05, 0),
    (16385, 2112, 13, 3, 0.0, 0),
    (14465, 2112, 64, 6, 0.05, 55),        # 114 x 9 = 1026 of them, the 114th row tile one token
    (14464, 2112, 64, 6, 0.05, 64),        # 113 x 9 = 1017: 128 x 128
    (65536, 320, 100, 4, 0.05, 4096),      # 512 x 2 = 1024
    (18725, 1792, 300, 8, 0.0, 0),         # 147 x 7 = 1029, whole column tiles, more experts than 256
    (4700, 7168, 129, 2, 0.0, 0),          # 37 x 28 = 1036
]


@pytest.mark.parametrize("flags", [L.MOE_SOFTMAX, L.MOE_SOFTMAX | L.MOE_GATES_RAW, L.MOE_GATES_RAW])
@pytest.mark.parametrize("T,H,E,k,alpha,seq", CASES)
def test_route_backward_of_a_large_batch(T, H, E, k, alpha, seq, flags):
    say(f"route backward, large, T={T} H={H} E={E} k={k} alpha={alpha} flags={flags}")
    softmax, raw = bool(flags & L.MOE_SOFTMAX), bool(flags & L.MOE_GATES_RAW)
    g = rng(231, T, H, E)
    x, w = grid(g, T, H, 1.0, 2.0 ** -3, 32), grid(g, E, H, 1.5 / np.sqrt(H), 2.0 ** -11, 61)
    s = oracle.affinity_softmax(x, w) if softmax else oracle.affinity(x, w)
    idx, _ = oracle.route(s, (g.uniform(-0.1, 0.1, E) / E).astype(np.float32), 1, 1, k, 1, 2.5)
    dg = g.standard_normal((T, k)).astype(np.float32)
    cfg = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 2.5, "bf16", "bf16")
    dx, dw, loss = backward(cfg, flags, x, w, s, idx, dg, alpha, seq)
    assert np.isfinite(dx).all()
    edge = np.arange(0, T, 128)
    rows = np.unique(np.concatenate([edge, edge[1:] - 1, np.arange((T - 1) // 128 * 128, T), g.integers(0, T, 300)]))
    rows = rows if len(rows) <= 700 else np.unique(np.concatenate([rows[:100], rows[-150:], g.choice(rows, 450)]))
    dlogit, dwr, lr = oracle.route_backward(x, np.eye(E), s, idx, dg, 2.5, alpha, seq, softmax, raw)
    tx, tw = bounds(x, w, s, idx, dg, alpha, softmax, raw, 2, rows)
    assert (np.abs(dx[rows] - dlogit[rows] @ w.astype(np.float64)) <= tx).all()
    assert (np.abs(dw - dwr) <= tw).all()
    assert abs(loss - lr) <= (T + E + 40) * EPS32 * abs(lr)
    _, again, _ = backward(cfg, flags, x, w, s, idx, dg, alpha, seq, with_dx=False)
    assert (again == dw).all()


def test_the_gradients_of_a_large_batch_repeat_their_bits():
    T, H, E, k = 16385, 2112, 256, 8
    say("route backward, large, repeated")
    g = rng(232)
    x, w = grid(g, T, H, 1.0, 2.0 ** -3, 32), grid(g, E, H, 1.5 / np.sqrt(H), 2.0 ** -11, 61)
    s = g.random((T, E)).astype(np.float32) / E
    idx = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    dg = g.standard_normal((T, k)).astype(np.float32)
    cfg = L.make_cfg(T, H, E, 1, 1, k, 0, 128, 1, 2.5, "bf16", "bf16")
    a, b = (backward(cfg, L.MOE_SOFTMAX, x, w, s, idx, dg, 0.05, 0) for _ in range(2))
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all() and a[2] == b[2]
