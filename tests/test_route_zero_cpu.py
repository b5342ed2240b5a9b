"""Tokens without any affinity (every logit -inf, or affinities that underflow) in the oracle's gradients."""
import numpy as np

import oracle
from oracle.backward import gate_backward
from workloads.inputs import rng


def test_a_token_without_affinities_adds_nothing():
    """The loss of a batch with such tokens is the loss of the others, scaled to the same sequence length, with the
    selections of all; their gradient is 0, the others' as in the formula."""
    g = rng(201)
    T, E, k, alpha = 12, 6, 2, 0.3
    s = g.random((T, E))
    s[[1, 7]] = 0
    idx = np.argsort(-s, axis=1, kind="stable")[:, :k]
    loss, ds = oracle.seq_balance_loss(s, idx, k, 4, alpha)
    want = 0.0
    for b in range(3):
        rows = range(4 * b, 4 * b + 4)
        f = np.zeros(E)
        P = np.zeros(E)
        for t in rows:
            f[idx[t]] += E / (k * 4)
            if t not in (1, 7):
                P += s[t] / s[t].sum() / 4
        want += alpha / 3 * (f * P).sum()
    assert np.isfinite(loss) and abs(loss - want) < 1e-12
    assert (ds[[1, 7]] == 0).all() and np.isfinite(ds).all()
    d = 1e-6
    for t, e in ((0, 0), (2, 3), (11, 5)):
        p = s.copy()
        p[t, e] += d
        m = s.copy()
        m[t, e] -= d
        num = (oracle.seq_balance_loss(p, idx, k, 4, alpha)[0] - oracle.seq_balance_loss(m, idx, k, 4, alpha)[0]) / (2 * d)
        assert abs(num - ds[t, e]) < 1e-7


def test_gates_without_affinities_have_no_gradient():
    s = np.array([[0.0, 0.0], [0.25, 0.5]])
    ds = gate_backward(s, np.ones((2, 2)) * [[3.0, 4.0]], 2.0)
    assert (ds[0] == 0).all()
    assert np.allclose(ds[1], 2 / 0.75 * (np.array([3.0, 4.0]) - (3 * 0.25 + 4 * 0.5) / 0.75))
