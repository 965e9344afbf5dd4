"""One token at a time over a paged cache, one plain fp64 definition each.

TEST INFRASTRUCTURE ONLY (see the package docstring): never imported by the
product path.  Arrays are numpy float64 unless stated; functions work on one
sequence (and one KV head where stated).  These are the standard definitions
(root-mean-square norm, rotary position embedding, softmax attention, eviction
by accumulated attention weight); the pages describe none of them.
"""
from __future__ import annotations

import numpy as np

from .steps import f64, gather_context, scale_for

__all__ = ["norm_rotate", "decode_attention", "evict_plan", "compact_rows", "cached_rows"]


def norm_rotate(x, pos: int, weight, eps: float, inv_freq, interleaved: bool) -> np.ndarray:
    """One head row x [d] at position pos: RMS norm with `weight` (None: no
    norm), then the rotation of the first 2 len(inv_freq) values."""
    y = f64(x).copy()
    if weight is not None:
        y = y * f64(weight) / np.sqrt(np.mean(y * y) + eps)
    f = np.zeros(0) if inv_freq is None else f64(inv_freq)
    n = len(f)
    for j in range(n):
        u, v = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
        a = float(pos) * f[j]
        y[u], y[v] = y[u] * np.cos(a) - y[v] * np.sin(a), y[v] * np.cos(a) + y[u] * np.sin(a)
    return y


def decode_attention(q_rows, K, V):
    """Rows q_rows [R][d] of one KV head over its cached tokens K, V [n][d].
    Returns (O [R][d], lse [R], weights [R][n]); n == 0: zeros and -inf."""
    q, K, V = f64(q_rows), f64(K), f64(V)
    R, d = q.shape
    if len(K) == 0:
        return np.zeros((R, d)), np.full(R, -np.inf), np.zeros((R, 0))
    S = (q @ K.T) * scale_for(d)
    m = S.max(axis=1, keepdims=True)
    E = np.exp(S - m)
    L = E.sum(axis=1, keepdims=True)
    P = E / L
    return P @ V, (m + np.log(L))[:, 0], P


def evict_plan(mass, pos, budget: int, n_first: int, n_recent: int):
    """One decision row of n tokens: (holes, fills), both ascending lists of
    indices.  A token is held when its position is below n_first or within
    n_recent of the largest; a held token ranks like +inf, a NaN mass like
    -inf; equal ranks to the lower index."""
    mass = np.asarray(mass, dtype=np.float64)
    n = len(mass)
    if n <= budget:
        return [], []
    pos = np.arange(n) if pos is None else np.asarray(pos, dtype=np.int64)
    held = (pos < n_first) | (pos > pos.max() - n_recent)
    key = np.where(np.isnan(mass), -np.inf, mass)
    key = np.where(held, np.inf, key)
    order = sorted(range(n), key=lambda t: (-key[t], t))
    stay = set(order[:budget])
    holes = [t for t in range(budget) if t not in stay]
    fills = [t for t in range(budget, n) if t in stay]
    return holes, fills


def compact_rows(pool, page_row, g: int, holes, fills, B: int) -> None:
    """KV head g's rows moved fill -> hole in `pool` [slots][H_kv][B][d], in
    place, through the page table row."""
    row = np.asarray(page_row, dtype=np.int64)
    moved = [pool[row[t // B], g, t % B].copy() for t in fills]
    for t, x in zip(holes, moved):
        pool[row[t // B], g, t % B] = x


def cached_rows(pool, page_row, g: int, n: int, B: int) -> np.ndarray:
    """The first n cached rows of KV head g, [n][d]."""
    return gather_context(f64(pool), np.asarray(page_row, dtype=np.int64), g, np.arange(n), B)
