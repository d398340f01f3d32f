"""Pins of the gated scan's oracle (CPU)."""

import numpy as np
import pytest

from oracle import gated_scan_oracle as go

GATES = ["sigmoid", "log", "decay"]


def inputs(n, d, gate, seed=0):
    r = np.random.default_rng(seed)
    g = r.normal(size=(n, d))
    g = {"sigmoid": g, "log": -np.abs(g), "decay": r.uniform(size=(n, d))}[gate]
    return r.normal(size=(n, d)), g, r.normal(size=(n, d)), r.normal(size=d), r.normal(size=d)


def test_two_tokens_by_hand():
    # decay: h1 = 1/2 * 4 + 3 = 5, h2 = 1/4 * 5 + 1 = 9/4
    x, g = np.array([[3.0], [1.0]]), np.array([[0.5], [0.25]])
    assert go.scan(x, g, "decay", np.array([4.0])).ravel().tolist() == [5.0, 2.25]
    # dy = (1, 2), dh_last = 1: G2 = 3, G1 = 1 + 3/4 = 7/4, dh0 = 7/8; dg = (7/4 * 4, 3 * 5)
    dx, dg, dh0 = go.scan_backward(x, g, np.array([[1.0], [2.0]]), "decay", np.array([4.0]), np.array([1.0]))
    assert dx.ravel().tolist() == [1.75, 3.0] and dg.ravel().tolist() == [7.0, 15.0] and dh0.tolist() == [0.875]
    # sigmoid(0) = 1/2: h = (0 + 2) / 2 = 1;  log: exp(log 1/2) = 1/2
    assert go.scan(np.array([[2.0]]), np.array([[0.0]]), "sigmoid").tolist() == [[1.0]]
    assert np.allclose(go.scan(x, np.log(g), "log", np.array([4.0])).ravel(), [5.0, 2.25], rtol=1e-15)


@pytest.mark.parametrize("gate", GATES)
def test_recurrence_is_the_explicit_sum(gate):
    x, g, _, h0, _ = inputs(9, 5, gate)
    for start in (None, h0):
        assert np.allclose(go.scan(x, g, gate, start), go.scan_bruteforce(x, g, gate, start), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("gate", GATES)
def test_gradients_are_the_differences(gate):
    n, d = 6, 3
    x, g, dy, h0, dl = inputs(n, d, gate, 3)
    got = go.scan_backward(x, g, dy, gate, h0, dl)

    def value(x, g, h0):
        y = go.scan(x, g, gate, h0)
        return (dy * y).sum() + (dl * y[-1]).sum()

    step = 1e-6
    for k, ref in enumerate(got):
        for i in np.ndindex(ref.shape):
            lo, hi = [x.copy(), g.copy(), h0.copy()], [x.copy(), g.copy(), h0.copy()]
            lo[k][i] -= step
            hi[k][i] += step
            assert abs((value(*hi) - value(*lo)) / (2 * step) - ref[i]) < 1e-8
