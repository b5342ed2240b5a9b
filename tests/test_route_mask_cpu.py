"""Experts out of service, on the CPU oracle: which of the two masks does what, through steps of the bias update."""
import numpy as np

import oracle
from oracle.balance import update_bias
from workloads.inputs import rng

INF = np.float32(np.inf)


def test_an_offset_alone_does_not_take_an_expert_out():
    """The ranking is by s + b: a bias above the others' affinities selects an expert whose affinity is 0."""
    logits = np.zeros((1, 8))
    logits[0, 0] = 20
    o = np.zeros(8, np.float32)
    o[5] = -INF
    s = oracle.affinity_softmax(logits, np.eye(8), o)
    assert s[0, 5] == 0
    bias = np.zeros(8, np.float32)
    bias[5] = 1e-3
    idx, w = oracle.route(s, bias, 1, 1, 2, 1, 1.0)
    assert idx.tolist() == [[0, 5]] and w[0, 1] == 0
    bias[5] = -INF
    idx, w = oracle.route(s, bias, 1, 1, 2, 1, 1.0)
    assert idx.tolist() == [[0, 1]]


def test_a_bias_of_minus_infinity_stays_and_keeps_the_expert_out():
    g = rng(211)
    T, E, G, M, k, topr, gamma = 40, 16, 4, 2, 3, 2, 0.05
    s = oracle.affinity_softmax(g.standard_normal((T, 8)), g.standard_normal((E, 8)))
    out = [3, 4, 5, 13]
    bias = np.zeros(E, np.float32)
    bias[out] = -INF
    for _ in range(50):
        idx, _ = oracle.route(s, bias, G, M, k, topr, 1.0)
        assert not np.isin(idx, out).any()
        counts = np.bincount(idx.reshape(-1), minlength=E)
        bias = update_bias(bias, counts, T, k, gamma)
        assert (bias[out] == -INF).all() and np.isfinite(np.delete(bias, out)).all()


def test_fewer_served_experts_than_slots():
    """The chosen groups' masked experts fill the slots, the lowest first, and never another group's."""
    s = np.full((1, 8), 0.125, np.float32)
    bias = np.zeros(8, np.float32)
    bias[[4, 6, 7]] = -INF                             # group 1 holds one served expert, group 0 four
    idx, _ = oracle.route(s, bias, 2, 1, 2, 1, 1.0)
    assert idx.tolist() == [[0, 1]]
    bias[:4] = -INF                                    # only expert 5 is left: group 1, whose masked ones follow it
    idx, _ = oracle.route(s, bias, 2, 1, 3, 1, 1.0)
    assert idx.tolist() == [[5, 4, 6]]
    bias[:] = 0
    bias[[0, 1, 2]] = -INF                             # one served expert in group 0: behind group 1 where two count
    s[0, 3] = 0.9
    assert oracle.route(s, bias, 2, 1, 2, 2, 1.0)[0].tolist() == [[4, 5]]
    assert oracle.route(s, bias, 2, 1, 2, 1, 1.0)[0].tolist() == [[3, 0]]
