"""Float64 oracle of the gated scan: a recurrence with a gate of its own for every token and channel.

Linear Attention notes §七 (the gated update S_t = G_t * S_{t-1} + ...), for a state of one vector:
h_t = a_t h_{t-1} + b_t, y_t = h_t, with a = sigmoid(g), b = (1 - a) x; a = exp(g), b = x; or a = g, b = x.
Pins (``tests/test_gated_scan_oracle.py``): the recurrence equals its explicit sum; hand-computed values; the
gradients equal central differences of the recurrence.
"""

from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def gates(g, gate):
    """a and the factor of x."""
    g = _f64(g)
    if gate == "decay":
        return g, np.ones_like(g)
    if gate == "log":
        return np.exp(g), np.ones_like(g)
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))


def scan(x, g, gate="sigmoid", h0=None, delta=0.0):
    """Outputs [N, D] of one sequence, token by token; h0 [D] or None.  With ``delta`` also a bound of what rounding
    does to them, where every gate, product and sum is off by at most delta of its terms' absolute values:
    e_t = |a_t| (e_{t-1} + delta m_{t-1}) + delta m_t, m the recurrence of absolute values."""
    a, take = gates(g, gate)
    b = take * _f64(x)
    h = np.zeros(a.shape[1]) if h0 is None else _f64(h0).copy()
    m, e = np.abs(h), np.zeros_like(h)
    y, bound = np.empty_like(b), np.empty_like(b)
    for t in range(len(a)):
        h = a[t] * h + b[t]
        e = np.abs(a[t]) * (e + delta * m)
        m = np.abs(a[t]) * m + np.abs(b[t])
        e = e + delta * m
        y[t], bound[t] = h, e
    return (y, bound) if delta else y


def scan_bruteforce(x, g, gate="sigmoid", h0=None):
    """The same outputs from the explicit sums of products of gates."""
    a, take = gates(g, gate)
    b = take * _f64(x)
    n = len(a)
    y = np.zeros_like(b)
    for t in range(n):
        for s in range(t + 1):
            y[t] += np.prod(a[s + 1:t + 1], axis=0) * b[s]
        if h0 is not None:
            y[t] += np.prod(a[:t + 1], axis=0) * _f64(h0)
    return y


def scan_backward(x, g, dy, gate="sigmoid", h0=None, dh_last=None, delta=0.0):
    """dx, dg, dh0 of sum(dy * y) + sum(dh_last * h_N) for one sequence: the chain rule through the recurrence.
    With ``delta`` also their rounding bounds (as in ``scan``), a triple behind the values."""
    a, take = gates(g, gate)
    x, dy = _f64(x), _f64(dy)
    n, d = a.shape
    start = np.zeros(d) if h0 is None else _f64(h0)
    y, ey = scan(x, g, gate, h0, delta or 1.0)
    before = np.concatenate([start[None], y[:-1]])
    eb = np.concatenate([np.zeros((1, d)), ey[:-1]])
    c = np.zeros(d) if dh_last is None else _f64(dh_last).copy()
    e, mc = np.zeros(d), np.abs(c)
    dx, dg, bx, bg = (np.empty_like(a) for _ in range(4))
    for t in reversed(range(n)):
        G, mG = dy[t] + c, np.abs(dy[t]) + mc
        eG = e + delta * mG
        inner = before[t] - x[t] if gate == "sigmoid" else before[t]
        mi = np.abs(before[t]) + np.abs(x[t]) if gate == "sigmoid" else np.abs(before[t])
        f = {"decay": np.ones(d), "log": a[t], "sigmoid": a[t] * take[t]}[gate]
        dx[t], dg[t] = take[t] * G, f * G * inner
        bx[t] = np.abs(take[t]) * (eG + 4 * delta * mG)
        bg[t] = np.abs(f) * (eG * mi + mG * (eb[t] + 6 * delta * mi))
        c = a[t] * G
        e = np.abs(a[t]) * (eG + delta * mG) + delta * np.abs(a[t]) * mG
        mc = np.abs(a[t]) * mG
    return ((dx, dg, c), (bx, bg, e)) if delta else (dx, dg, c)
