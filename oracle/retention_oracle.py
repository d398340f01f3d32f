"""Float64 oracle of the retention operators: linear attention with a decay for each head.

Linear Attention notes §七 (RetNet): S_t = gamma S_{t-1} + phi(k_t) v_t^T, out_t = phi(q_t) S_t, with a
decay gamma_h of its own for each head and a scale on the output.  Pins (``tests/test_retention_oracle.py``):
the recurrence equals its brute force; a hand-computed two-token value; the gradients equal central
differences of the recurrence.
"""

from __future__ import annotations

import numpy as np

FEATURES = {
    "identity": (lambda x: x, lambda x: np.ones_like(x)),
    "elu1": (lambda x: np.where(x > 0, x + 1, np.exp(np.minimum(x, 0))),
             lambda x: np.where(x > 0, 1.0, np.exp(np.minimum(x, 0)))),
    "relu": (lambda x: np.maximum(x, 0.0), lambda x: (x > 0).astype(np.float64)),
    "exp": (np.exp, np.exp),
}


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def retention(q, k, v, gamma, scale=1.0, feature="identity", state=None, magnitude=False):
    """Outputs and final state of one sequence, token by token: q, k, v [H, N, d], gamma [H], state
    [H, d, d] or None.  With ``magnitude`` every term is taken by its absolute value: the scale that
    rounding errors of the sums go by."""
    q, k, v, g = _f64(q), _f64(k), _f64(v), _f64(gamma)[:, None, None]
    f = FEATURES[feature][0]
    h, n, d = q.shape
    s = np.zeros((h, d, d)) if state is None else _f64(state).copy()
    fq, fk = f(q), f(k)
    if magnitude:
        fq, fk, v, s, scale = np.abs(fq), np.abs(fk), np.abs(v), np.abs(s), abs(scale)
    y = np.empty_like(q)
    for t in range(n):
        s = g * s + fk[:, t, :, None] * v[:, t, None, :]
        y[:, t] = scale * np.matmul(fq[:, t, None, :], s)[:, 0]
    return y, s


def retention_bruteforce(q, k, v, gamma, scale=1.0, feature="identity", state=None):
    """The same outputs from the explicit N x N matrix gamma^(t-s) phi(q_t).phi(k_s), s <= t."""
    q, k, v, gamma = _f64(q), _f64(k), _f64(v), _f64(gamma)
    f = FEATURES[feature][0]
    n = q.shape[1]
    i = np.arange(n)
    age = i[:, None] - i[None, :]
    w = np.where(age >= 0, gamma[:, None, None] ** np.maximum(age, 0), 0.0)
    y = (w * (f(q) @ f(k).transpose(0, 2, 1))) @ v
    if state is not None:
        y = y + (gamma[:, None] ** (i + 1))[..., None] * (f(q) @ _f64(state))
    return scale * y


def retention_backward(q, k, v, gamma, dy, scale=1.0, feature="identity", magnitude=False):
    """dq, dk, dv of sum(dy * y) for one sequence from a zero state: the chain rule through the
    recurrence, S_t forwards, G_t = gamma G_{t+1} + scale phi(q_t) dy_t^T backwards."""
    q, k, v, dy, g = _f64(q), _f64(k), _f64(v), _f64(dy), _f64(gamma)[:, None, None]
    f, df = FEATURES[feature]
    h, n, d = q.shape
    fq, fk, dfq, dfk = f(q), f(k), df(q), df(k)
    if magnitude:
        fq, fk, v, dy, scale = np.abs(fq), np.abs(fk), np.abs(v), np.abs(dy), abs(scale)
    dq, dk, dv = np.empty_like(q), np.empty_like(q), np.empty_like(q)
    s = np.zeros((h, d, d))
    for t in range(n):
        s = g * s + fk[:, t, :, None] * v[:, t, None, :]
        dq[:, t] = dfq[:, t] * scale * np.matmul(s, dy[:, t, :, None])[..., 0]
    gs = np.zeros((h, d, d))
    for t in reversed(range(n)):
        gs = g * gs + scale * fq[:, t, :, None] * dy[:, t, None, :]
        dk[:, t] = dfk[:, t] * np.matmul(gs, v[:, t, :, None])[..., 0]
        dv[:, t] = np.matmul(fk[:, t, None, :], gs)[:, 0]
    return dq, dk, dv
