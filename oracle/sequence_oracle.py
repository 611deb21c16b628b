"""float64 NumPy oracle of the sequence operators: rotary positions, and linear attention with a
decay per head, token by token (the recurrence itself) with the gradients of that recurrence.
Independent of the package: it shares no code or constants with it."""
from __future__ import annotations

import math

import numpy as np


def rotary(x, positions, freq, scale=1.0, interleaved=False, inverse=False):
    """x [..., n, D]; positions [n, R/2] (each pair's own) or [n]; freq [R/2]."""
    x = np.asarray(x, np.float64)
    freq = np.asarray(freq, np.float64)
    R = 2 * len(freq)
    pos = np.asarray(positions, np.float64)
    a = (pos[:, None] if pos.ndim == 1 else pos) * freq * (-1.0 if inverse else 1.0)
    c, s = scale * np.cos(a), scale * np.sin(a)
    i1 = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
    i2 = i1 + 1 if interleaved else i1 + R // 2
    y = x.copy()
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def decay_forward(q, k, v, g, S0=None, scale=1.0):
    """One head: q, k, v [n, D] -> (out [n, D], state after the last row [D, D])."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, D = q.shape
    S = np.zeros((D, D)) if S0 is None else np.array(S0, np.float64)
    lam = math.exp(g)
    out = np.zeros((n, D))
    for i in range(n):
        S = lam * S + np.outer(k[i], v[i])
        out[i] = scale * (q[i] @ S)
    return out, S


def decay_backward(q, k, v, g, dout, S0=None, dS=None, scale=1.0):
    """Gradients of sum(dout * out) + sum(dS * last state): the recurrence run backwards.
    Returns dq, dk, dv, dS0."""
    q, k, v, dout = (np.asarray(x, np.float64) for x in (q, k, v, dout))
    n, D = q.shape
    lam = math.exp(g)
    S = np.zeros((D, D)) if S0 is None else np.array(S0, np.float64)
    dq = np.zeros((n, D))
    for i in range(n):
        S = lam * S + np.outer(k[i], v[i])
        dq[i] = scale * (S @ dout[i])
    R = np.zeros((D, D)) if dS is None else np.array(dS, np.float64)
    dk, dv = np.zeros((n, D)), np.zeros((n, D))
    for i in range(n - 1, -1, -1):
        R = R + scale * np.outer(q[i], dout[i])
        dk[i], dv[i] = R @ v[i], R.T @ k[i]
        R = lam * R
    return dq, dk, dv, R
