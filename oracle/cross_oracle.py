"""Float64 oracle of linear cross attention: queries that read another sequence's keys and values.

Linear Attention notes §三 with the keys and values of an encoder: S = sum phi(k_j) v_j^T, z = sum phi(k_j),
y_t = phi(q_t) S / (phi(q_t) . z + eps), or without the normaliser.  Pins (``tests/test_cross_oracle.py``): the sums
equal the explicit weights over all pairs of tokens; a hand-computed value; the gradients equal central differences.
"""

from __future__ import annotations

import numpy as np

from .retention_oracle import FEATURES


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def states(k, v, feature="elu1"):
    """S [Hk, d, d] and z [Hk, d] of k, v [Hk, N, d]."""
    fk = FEATURES[feature][0](_f64(k))
    return np.matmul(fk.transpose(0, 2, 1), _f64(v)), fk.sum(1)


def _inverse(den):
    return np.divide(1.0, den, out=np.zeros_like(den), where=den != 0)


def read(q, S, z, feature="elu1", normalise=True, eps=1e-6):
    """y [H, N, d] of q [H, N, d]; query head h reads head h // (H / Hk)."""
    per = len(q) // len(S)
    fq = FEATURES[feature][0](_f64(q))
    num = np.matmul(fq, np.repeat(_f64(S), per, 0))
    if not normalise:
        return num
    return num * _inverse(np.matmul(fq, np.repeat(_f64(z), per, 0)[..., None]) + eps)


def bruteforce(q, k, v, feature="elu1", normalise=True, eps=1e-6):
    """The same outputs from the explicit weights phi(q_t) . phi(k_j)."""
    per = len(q) // len(k)
    f = FEATURES[feature][0]
    w = np.matmul(f(_f64(q)), f(np.repeat(_f64(k), per, 0)).transpose(0, 2, 1))
    y = np.matmul(w, np.repeat(_f64(v), per, 0))
    return y * _inverse(w.sum(-1, keepdims=True) + eps) if normalise else y


def backward(q, k, v, dy, feature="elu1", normalise=True, eps=1e-6, S=None, z=None):
    """dq, dk, dv of sum(dy * y): the chain rule through read and states (S, z: theirs unless given)."""
    f, df = FEATURES[feature]
    q, k, v, dy = _f64(q), _f64(k), _f64(v), _f64(dy)
    hk, per = len(k), len(q) // len(k)
    S, z = states(k, v, feature) if S is None else (_f64(S), _f64(z))
    fq, fk = f(q), f(k)
    Sq, zq = np.repeat(S, per, 0), np.repeat(z, per, 0)
    u = np.matmul(dy, Sq.transpose(0, 2, 1))
    if normalise:
        inv = _inverse(np.matmul(fq, zq[..., None]) + eps)
        dden = -(fq * u).sum(-1, keepdims=True) * inv * inv
    else:
        inv, dden = np.ones(fq.shape[:2] + (1,)), np.zeros(fq.shape[:2] + (1,))
    dq = df(q) * (u * inv + dden * zq[:, None])
    dS = np.matmul((fq * inv).transpose(0, 2, 1), dy).reshape(hk, per, *S.shape[1:]).sum(1)
    dz = (fq * dden).sum(1).reshape(hk, per, -1).sum(1)
    dk = df(k) * (np.matmul(v, dS.transpose(0, 2, 1)) + dz[:, None])
    return dq, dk, np.matmul(fk, dS)


def magnitudes(q, k, v, dy, feature="elu1", normalise=True, eps=1e-6):
    """For each of S, z, y, dq, dk, dv the sum of its terms' absolute values: the scale that rounding errors of
    operands and sums go by (the denominators, sums of terms >= 0, are taken as they are)."""
    f, df = FEATURES[feature]
    q, k, v, dy = _f64(q), _f64(k), _f64(v), np.abs(_f64(dy))
    hk, per = len(k), len(q) // len(k)
    fq, fk, v = np.abs(f(q)), np.abs(f(k)), np.abs(v)
    S, z = np.matmul(fk.transpose(0, 2, 1), v), fk.sum(1)
    Sq, zq = np.repeat(S, per, 0), np.repeat(z, per, 0)
    inv = _inverse(np.matmul(fq, zq[..., None]) + eps) if normalise else np.ones(fq.shape[:2] + (1,))
    y = np.matmul(fq, Sq) * inv
    u = np.matmul(dy, Sq.transpose(0, 2, 1))
    dden = (fq * u).sum(-1, keepdims=True) * inv * inv * (1.0 if normalise else 0.0)
    dq = np.abs(df(q)) * (u * inv + dden * zq[:, None])
    dS = np.matmul((fq * inv).transpose(0, 2, 1), dy).reshape(hk, per, *S.shape[1:]).sum(1)
    dz = (fq * dden).sum(1).reshape(hk, per, -1).sum(1)
    dk = np.abs(df(k)) * (np.matmul(v, dS.transpose(0, 2, 1)) + dz[:, None])
    return S, z, y, dq, dk, np.matmul(fk, dS)
