"""Attention over a cache and eviction by accumulated weight in 64 bits, row by
row from the definitions, on numpy arrays. Shares no code with the library.

A slice is k, v [n, d]; the query of new token i of n_new sits at row
r = n - n_new + i and sees row j when j <= r and (window == 0 or j < n_sink or
j > r - window)."""
from __future__ import annotations

import numpy as np


def visible(r: int, n: int, n_sink: int, window: int) -> np.ndarray:
    j = np.arange(n)
    seen = j <= r
    if window > 0:
        seen &= (j < n_sink) | (j > r - window)
    return seen


def attend(q, k, v, r: int, scale: float, n_sink: int = 0, window: int = 0):
    """One query [d] at row r: (out [d], lse, weights [n])."""
    n, d = k.shape
    w = np.zeros(n)
    idx = np.nonzero(visible(r, n, n_sink, window))[0]
    if idx.size == 0:
        return np.zeros(d), -np.inf, w
    x = scale * (k[idx].astype(np.float64) @ q.astype(np.float64))
    m = x.max()
    e = np.exp(x - m)
    w[idx] = e / e.sum()
    return w[idx] @ v[idx].astype(np.float64), m + np.log(e.sum()), w


def evict(mass, n: int, n_prompt: int, n_recent: int, budget: int):
    """Kept rows, ascending, of one slice: protected rows and the largest masses (ties: low row)."""
    if n <= budget:
        return np.arange(n)
    cand = list(range(n_prompt, n - n_recent))
    cand.sort(key=lambda j: (-float(mass[j]), j))
    best = cand[: budget - n_prompt - n_recent]
    return np.array(sorted(list(range(n_prompt)) + best + list(range(n - n_recent, n))), dtype=np.int64)
