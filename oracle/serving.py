"""The residual stream's norm, in the input's type or in 8 bits, and the gated delta rule, fp64 oracle (test
infrastructure only). Plain loops over tokens and heads, straight from the formulas.

The gated delta rule is the fast weight of TTT-Linear at a mini-batch of one token (TTT layers page: the
delta rule) with a decay of the state before each token.
"""
from __future__ import annotations

import math

import numpy as np

f64 = np.float64


def e4m3_values():
    """The value of each of the 256 codes: sign, 4 bits of exponent (bias 7), 3 of fraction; exponent 0 holds
    multiples of 2^-9, and only the code with all other bits set is NaN (there are no infinities)."""
    out = np.zeros(256, f64)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = -x if c & 128 else x
    return out


def add_rms_norm(X, R, weight, eps):
    """(y, h): h = X + R (R None: X), y = h / sqrt(mean(h^2) + eps) * weight, row by row."""
    H = np.asarray(X, f64) + (0.0 if R is None else np.asarray(R, f64))
    Y = np.empty_like(H)
    for n, h in enumerate(H):
        Y[n] = h / math.sqrt((h * h).mean() + eps) * (1.0 if weight is None else np.asarray(weight, f64))
    return Y, H


def e4m3_scales(Y, group=0):
    """max(max |y| / 448, 2^-126) of each row, or of each `group` channels."""
    N, D = Y.shape
    top = np.abs(Y).reshape(N, -1, group or D).max(axis=-1)
    s = np.maximum(top / 448, 2.0 ** -126)
    return s if group else s[:, 0]


def gated_delta(Q, K, V, g, beta, state, scale, eps=None):
    """One sequence, token by token: Q, K [T, Hk, dk], V [T, Hv, dv], g, beta [T, Hv], state [Hv, dk, dv] or
    None; eps None: q and k as they are. Returns (O [T, Hv, dv], the last state, and the same two with each
    product replaced by its size and each difference by a sum: what roundings are measured against)."""
    Q, K, V, g, beta = (np.asarray(x, f64) for x in (Q, K, V, g, beta))
    T, Hk, dk = Q.shape
    Hv, dv = V.shape[1:]
    W = np.zeros((Hv, dk, dv)) if state is None else np.array(state, f64)
    A = np.abs(W)
    O, B = np.zeros((T, Hv, dv)), np.zeros((T, Hv, dv))
    for t in range(T):
        for h in range(Hv):
            q, k = Q[t, h // (Hv // Hk)], K[t, h // (Hv // Hk)]
            if eps is not None:
                q, k = (x / math.sqrt((x * x).sum() + eps) for x in (q, k))
            keep = math.exp(g[t, h])
            W[h], A[h] = keep * W[h], keep * A[h]
            u = beta[t, h] * (V[t, h] - k @ W[h])
            a = abs(beta[t, h]) * (np.abs(V[t, h]) + np.abs(k) @ A[h])
            W[h] += np.outer(k, u)
            A[h] += np.outer(np.abs(k), a)
            O[t, h], B[t, h] = scale * (q @ W[h]), abs(scale) * (np.abs(q) @ A[h])
    return O, W, B, A
