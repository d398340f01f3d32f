"""Pins of the retention oracle and of what its tolerances rest on (CPU)."""

import numpy as np
import pytest

from oracle import retention_oracle as ro

RNG = np.random.default_rng


def _inputs(seed, h, n, d):
    r = RNG(seed)
    return [r.standard_normal((h, n, d)) for _ in range(4)] + [np.array([0.0, 1.0, 0.5, 0.97])[:h]]


@pytest.mark.parametrize("feature", list(ro.FEATURES))
@pytest.mark.parametrize("n", [1, 2, 9, 40])
def test_recurrence_equals_brute_force(feature, n):
    q, k, v, s, gamma = _inputs(n, 4, n, 5)
    state = RNG(5).standard_normal((4, 5, 5))
    for st in (None, state):
        y, _ = ro.retention(q, k, v, gamma, 0.7, feature, st)
        np.testing.assert_allclose(y, ro.retention_bruteforce(q, k, v, gamma, 0.7, feature, st), rtol=1e-12, atol=1e-12)


def test_two_tokens_by_hand():
    """d = 1: S_1 = 2*3 = 6, y_1 = 0.5*(4*6) = 12; S_2 = 0.5*6 + 1*10 = 13, y_2 = 0.5*(-2*13) = -13."""
    one = lambda *x: np.array(x, float).reshape(1, 2, 1)
    y, s = ro.retention(one(4, -2), one(2, 1), one(3, 10), [0.5], scale=0.5)
    assert y.ravel().tolist() == [12.0, -13.0] and s.ravel().tolist() == [13.0]


def test_a_split_sequence_continues_from_its_state():
    q, k, v, _, gamma = _inputs(3, 4, 20, 6)
    y, s = ro.retention(q, k, v, gamma)
    y1, s1 = ro.retention(q[:, :7], k[:, :7], v[:, :7], gamma)
    y2, s2 = ro.retention(q[:, 7:], k[:, 7:], v[:, 7:], gamma, state=s1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, rtol=1e-13, atol=1e-13)
    np.testing.assert_allclose(s2, s, rtol=1e-13, atol=1e-13)


@pytest.mark.parametrize("feature", ["identity", "elu1", "exp", "relu"])
def test_gradients_equal_central_differences(feature):
    h, n, d, eps = 2, 6, 3, 1e-6
    r = RNG(11)
    q, k, v, dy = (r.standard_normal((h, n, d)) for _ in range(4))
    if feature == "relu":  # away from its corner
        q, k = (np.where(np.abs(x) < 0.01, 0.5, x) for x in (q, k))
    gamma = np.array([0.9, 0.4])
    grads = ro.retention_backward(q, k, v, gamma, dy, 0.8, feature)
    for x, gx in zip((q, k, v), grads):
        for idx in np.ndindex(x.shape):
            old = x[idx]
            x[idx] = old + eps
            up = (dy * ro.retention(q, k, v, gamma, 0.8, feature)[0]).sum()
            x[idx] = old - eps
            down = (dy * ro.retention(q, k, v, gamma, 0.8, feature)[0]).sum()
            x[idx] = old
            assert abs((up - down) / (2 * eps) - gx[idx]) <= 1e-7 * (1 + abs(gx[idx]))


def test_a_mistake_in_the_oracle_is_seen():
    """One decay for all heads, a decay after the update, a transposed state: each differs."""
    q, k, v, _, gamma = _inputs(8, 3, 12, 4)
    y = ro.retention_bruteforce(q, k, v, gamma)
    assert np.abs(ro.retention(q, k, v, np.full(3, gamma.mean()))[0] - y).max() > 1e-2
    late = np.concatenate([np.zeros((3, 1, 4)), k[:, :-1]], 1), np.concatenate([np.zeros((3, 1, 4)), v[:, :-1]], 1)
    assert np.abs(ro.retention(q, *late, gamma)[0] - y).max() > 1e-2
    assert np.abs(ro.retention(q, v, k, gamma)[0] - y).max() > 1e-2
