"""Norm and rotation of queries and keys, causal attention over packed sequences and over a paged
cache, fp64 oracle (test infrastructure only).

The attention that In-Place TTT keeps beside the fast weights (In-Place TTT page, sections 3 and
7: full or sliding-window attention handles what lies inside a chunk). Plain loops over sequences,
queries and heads, straight from the formulas.
"""
from __future__ import annotations

import math

import numpy as np

f64 = np.float64


def rope_frequencies(rot, base, scaling=None, factor=1.0, original_length=0, beta_fast=32.0,
                     beta_slow=1.0):
    """(inv_freq [rot / 2], rope_scale), pair by pair."""
    out, scale = [], 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    if scaling == "yarn":
        def pair(turns):  # where base^(-2 j / rot) * original_length = 2 pi turns
            return rot / 2 * math.log(original_length / (2 * math.pi * turns)) / math.log(base)
        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), rot - 1)
        if high <= low:
            high = low + 0.001
        scale = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    for j in range(rot // 2):
        f = base ** (-2 * j / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            ramp = min(max((j - low) / (high - low), 0), 1)
            f = f / factor * ramp + f * (1 - ramp)
        out.append(f)
    return np.array(out, f64), scale


def norm_rope(X, weight, eps, pos, inv_freq, layout, rope_scale):
    """X [N, H, dh] -> the same, normed (where a weight is given) and rotated."""
    Y = np.array(X, f64)
    if weight is not None:
        ms = (Y * Y).mean(axis=-1, keepdims=True)
        Y = Y / np.sqrt(ms + eps) * np.asarray(weight, f64)
    half = len(inv_freq)
    for t, p in enumerate(pos):
        for j in range(half):
            a, b = (j, j + half) if layout == "half" else (2 * j, 2 * j + 1)
            ang = float(p) * float(inv_freq[j])
            c, s = rope_scale * math.cos(ang), rope_scale * math.sin(ang)
            xa, xb = Y[t, :, a].copy(), Y[t, :, b].copy()
            Y[t, :, a] = xa * c - xb * s
            Y[t, :, b] = xa * s + xb * c
    return Y


def attend(q, K, V, scale):
    """One query over its visible keys: (o, lse, sum of weight * |v|)."""
    if len(K) == 0:
        return np.zeros(V.shape[-1]), -np.inf, np.zeros(V.shape[-1])
    x = scale * (K @ q)
    m = x.max()
    w = np.exp(x - m)
    n = w.sum()
    return w @ V / n, m + math.log(n), w @ np.abs(V) / n


def packed(Q, K, V, cu_q, cu_k, scale, window=0):
    """Q [Nq, Hq, dh], K, V [Nk, Hkv, dh]: (O, lse, the sums of weight * |v|); rows of no sequence
    are NaN."""
    Q, K, V = (np.asarray(x, f64) for x in (Q, K, V))
    Nq, Hq, dh = Q.shape
    G = Hq // K.shape[1]
    O = np.full((Nq, Hq, dh), np.nan)
    A = np.full((Nq, Hq, dh), np.nan)
    L = np.full((Nq, Hq), np.nan)
    for s in range(len(cu_q) - 1):
        lq, lk = cu_q[s + 1] - cu_q[s], cu_k[s + 1] - cu_k[s]
        for i in range(lq):
            last = i + lk - lq
            first = max(0, last - window + 1) if window else 0
            ks = slice(cu_k[s] + first, cu_k[s] + max(first, last + 1))
            for h in range(Hq):
                t = cu_q[s] + i
                O[t, h], L[t, h], A[t, h] = attend(Q[t, h], K[ks, h // G], V[ks, h // G], scale)
    return O, L, A


def decode(Q, Kc, Vc, table, lengths, page, scale, window=0):
    """Q [S, Hq, dh], caches [n_slots, Hkv, dh]: as packed, one query per sequence."""
    Q, Kc, Vc = (np.asarray(x, f64) for x in (Q, Kc, Vc))
    S, Hq, dh = Q.shape
    G = Hq // Kc.shape[1]
    n_pages = len(Kc) // page
    O, A, L = np.zeros((S, Hq, dh)), np.zeros((S, Hq, dh)), np.zeros((S, Hq))
    for s in range(S):
        n = min(max(int(lengths[s]), 0), table.shape[1] * page)
        first = max(0, n - window) if window else 0
        rows = [int(table[s, j // page]) * page + j % page for j in range(first, n)
                if 0 <= table[s, j // page] < n_pages]
        for h in range(Hq):
            O[s, h], L[s, h], A[s, h] = attend(Q[s, h], Kc[rows, h // G], Vc[rows, h // G], scale)
    return O, L, A
