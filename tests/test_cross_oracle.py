"""Pins of the cross attention oracle (CPU)."""

import numpy as np
import pytest

from oracle import cross_oracle as co

CASES = [("elu1", True, 1e-6), ("elu1", True, 0.3), ("exp", True, 1e-6), ("relu", True, 0.2), ("identity", False, 0.0),
         ("elu1", False, 0.0)]


def inputs(H=4, Hk=2, nq=5, nk=7, d=3, seed=0):
    r = np.random.default_rng(seed)
    return r.normal(size=(H, nq, d)), r.normal(size=(Hk, nk, d)), r.normal(size=(Hk, nk, d)), r.normal(size=(H, nq, d))


def test_one_query_of_two_tokens_by_hand():
    # identity features of q = 2, k = (1, 3), v = (5, -1): S = 5 - 3 = 2, z = 4
    q, k, v = np.array([[[2.0]]]), np.array([[[1.0], [3.0]]]), np.array([[[5.0], [-1.0]]])
    S, z = co.states(k, v, "identity")
    assert S.ravel().tolist() == [2.0] and z.ravel().tolist() == [4.0]
    assert co.read(q, S, z, "identity", normalise=False).ravel().tolist() == [4.0]
    # with it: 4 / (8 + 2) = 0.4;  dy = 10: u = 20, dden = -(2 * 20) / 100 = -0.4, dq = 20 / 10 - 0.4 * 4 = 0.4
    assert np.isclose(co.read(q, S, z, "identity", eps=2.0).item(), 0.4)
    dq, dk, dv = co.backward(q, k, v, np.array([[[10.0]]]), "identity", eps=2.0)
    # dS = 2 / 10 * 10 = 2, dz = -0.8: dk = 2 v - 0.8, dv = 2 k
    assert np.allclose(dq.ravel(), [0.4]) and np.allclose(dk.ravel(), [9.2, -2.8]) and np.allclose(dv.ravel(), [2.0, 6.0])


@pytest.mark.parametrize("feature,normalise,eps", CASES)
def test_sums_are_the_explicit_weights(feature, normalise, eps):
    q, k, v, _ = inputs()
    S, z = co.states(k, v, feature)
    assert np.allclose(co.read(q, S, z, feature, normalise, eps), co.bruteforce(q, k, v, feature, normalise, eps), rtol=1e-12)


def test_no_tokens_and_no_eps_give_zeros():
    q, k, v, dy = inputs()
    k0, v0 = k[:, :0], v[:, :0]
    S, z = co.states(k0, v0)
    assert not co.read(q, S, z, eps=0.0).any() and not any(g.any() for g in co.backward(q, k0, v0, dy, eps=0.0))


@pytest.mark.parametrize("feature,normalise,eps", CASES)
def test_gradients_are_the_differences(feature, normalise, eps):
    q, k, v, dy = inputs(seed=4)
    got = co.backward(q, k, v, dy, feature, normalise, eps)
    step = 1e-6
    for n, ref in enumerate(got):
        for i in np.ndindex(ref.shape):
            lo, hi = [q.copy(), k.copy(), v.copy()], [q.copy(), k.copy(), v.copy()]
            lo[n][i] -= step
            hi[n][i] += step
            diff = (dy * (co.bruteforce(*hi, feature, normalise, eps) - co.bruteforce(*lo, feature, normalise, eps))).sum()
            assert abs(diff / (2 * step) - ref[i]) < 1e-6 * (1 + abs(ref[i]))
