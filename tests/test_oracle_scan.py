"""Pins of the recurrence's oracle: the sequential scan of every root-to-leaf path, central finite
differences of a random loss, and the routed states of the hybrid oracle."""
import numpy as np
import pytest

import oracle
from oracle import scan as osc
from workloads import random_tree


def _inputs(N, n, C, kind, seed):
    rng = np.random.default_rng(seed)
    gate = rng.normal(1.0, 2.0, (N, C)) if kind == "sigmoid" else -np.exp(rng.normal(-1.0, 1.0, (N, C)))
    return gate, rng.normal(size=(N, C)), rng.normal(size=(n, C)), rng.normal(size=(N, C)), rng.normal(size=(n, C))


@pytest.mark.parametrize("kind", ["sigmoid", "log"])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_equals_the_sequential_scan_of_every_path(kind, seed):
    parent, node_len = random_tree(seed, 25, max_len=7, zero_prob=0.25, n_roots=1 + seed)
    p = oracle.plan(parent, node_len)
    gate, x, init, _, _ = _inputs(p["n_tokens"], len(parent), 3, kind, seed)
    got = osc.scan(parent, node_len, gate, x, kind, init=init, p=p)
    for path in p["paths"]:
        h = None
        for v in path:
            if node_len[v] and h is None:
                h = init[v].copy()
            for t in range(p["tok_start"][v], p["tok_start"][v] + node_len[v]):
                if kind == "sigmoid":
                    a = 1 / (1 + np.exp(-gate[t]))
                    h = a * h + (1 - a) * x[t]
                else:
                    h = np.exp(gate[t]) * h + x[t]
                np.testing.assert_allclose(got["y"][t], h, rtol=1e-12, atol=1e-12)
            np.testing.assert_allclose(got["final"][v], h if node_len[v] else 0 * x[0], rtol=1e-12, atol=1e-12)


def test_a_node_starts_from_the_state_that_is_routed_to_it():
    parent, node_len = random_tree(7, 30, max_len=5, zero_prob=0.3, n_roots=2)
    p = oracle.plan(parent, node_len)
    gate, x, _, _, _ = _inputs(p["n_tokens"], 30, 4, "sigmoid", 3)
    got = osc.scan(parent, node_len, gate, x, "sigmoid", p=p)
    init = oracle.route_states(parent, node_len, got["final"])
    for v in range(30):
        if node_len[v]:
            t = p["tok_start"][v]
            a = 1 / (1 + np.exp(-gate[t]))
            np.testing.assert_allclose(got["y"][t], a * init[v] + (1 - a) * x[t], rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["sigmoid", "log"])
def test_gradients_against_finite_differences(kind):
    parent, node_len = random_tree(11, 9, max_len=4, zero_prob=0.2, n_roots=2)
    N = int(node_len.sum())
    gate, x, init, dy, dfin = _inputs(N, 9, 2, kind, 5)

    def loss(g, xx, ii):
        o = osc.scan(parent, node_len, g, xx, kind, init=ii)
        return (o["y"] * dy).sum() + (o["final"] * dfin).sum()

    got = osc.scan(parent, node_len, gate, x, kind, init=init, dy=dy, d_final=dfin)
    for name, arr, args in (("dgate", gate, 0), ("dx", x, 1), ("d_init", init, 2)):
        for i in np.ndindex(arr.shape):
            v = [gate, x, init]
            hi, lo = arr.copy(), arr.copy()
            hi[i] += 1e-6
            lo[i] -= 1e-6
            v[args] = hi
            up = loss(*v)
            v[args] = lo
            np.testing.assert_allclose(got[name][i], (up - loss(*v)) / 2e-6, rtol=2e-5, atol=2e-7)


def test_log_gate_is_held_at_zero():
    gate = np.array([[0.5], [0.0], [-1.0]])
    o = osc.scan([-1], [3], gate, np.ones((3, 1)), "log", dy=np.ones((3, 1)))
    np.testing.assert_allclose(o["y"][:, 0], [1, 2, 2 * np.exp(-1) + 1])
    assert o["dgate"][0, 0] == 0 and o["dgate"][1, 0] != 0
