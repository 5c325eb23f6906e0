"""Attention of new tokens over a paged cache, the residual stream's norm, in the input's type or in 8 bits,
and the gated delta rule, fp64 oracle (test infrastructure only). Plain loops over tokens and heads,
straight from the formulas.

The gated delta rule is the fast weight of TTT-Linear at a mini-batch of one token (TTT layers page: the
delta rule) with a decay of the state before each token.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import attend

f64 = np.float64


def paged(Q, Kc, Vc, cu_q, table, lengths, page, scale, window=0, rows=None):
    """Q [Nq, Hq, dh], caches [n_slots, Hkv, dh]: (O, lse, the sums of weight * |v|), of the queries `rows`
    (None: all); other rows, and those of no sequence, are NaN. Tokens of a page that is not there are left
    out."""
    Q, Kc, Vc = (np.asarray(x, f64) for x in (Q, Kc, Vc))
    Nq, Hq, dh = Q.shape
    G, n_pages = Hq // Kc.shape[1], len(Kc) // page
    O, A, L = (np.full(s, np.nan) for s in ((Nq, Hq, dh), (Nq, Hq, dh), (Nq, Hq)))
    for s in range(len(cu_q) - 1):
        lq, n = cu_q[s + 1] - cu_q[s], min(max(int(lengths[s]), 0), table.shape[1] * page)
        for i in range(lq):
            t, last = cu_q[s] + i, i + n - lq
            if rows is not None and t not in rows:
                continue
            first = max(0, last - window + 1) if window else 0
            at = [int(table[s, j // page]) * page + j % page for j in range(first, last + 1)
                  if 0 <= table[s, j // page] < n_pages]
            for h in range(Hq):
                O[t, h], L[t, h], A[t, h] = attend(Q[t, h], Kc[at, h // G], Vc[at, h // G], scale)
    return O, L, A


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
