"""Plain 64-bit definitions of the filters, a row at a time, for the tests."""
from __future__ import annotations

import math

import numpy as np


def usable(row, T, k, p, m):
    finite = row[np.isfinite(row)]
    return (not np.isnan(row).any() and not (row == np.inf).any() and finite.size > 0 and
            (T == 0 or (np.isfinite(T) and T >= np.finfo(np.float32).tiny)) and k >= 0 and 0 <= p <= 1 and 0 <= m <= 1)


def kept_of(row, T, k=0, p=1.0, m=0.0):
    """Indices of the kept tokens in the order of the draw, and their weights; None for an unusable row."""
    row = np.asarray(row, np.float64)
    if not usable(row, T, k, p, m):
        return None
    order = np.argsort(-row, kind="stable")
    order = order[row[order] > -np.inf]
    if T == 0:
        return order[:1], np.ones(1)
    with np.errstate(over="ignore"):
        w = np.exp((row[order] - row[order[0]]) / np.float64(T))
    if m > 0:
        n = int((w >= m).sum())
        order, w = order[:n], w[:n]
    if k > 0:
        order, w = order[:k], w[:k]
    if p < 1:
        mass = np.cumsum(w)
        n = max(1, int((mass < p * mass[-1]).sum()) + 1)
        order, w = order[:n], w[:n]
    return order, w


def draw_of(row, u, T, k=0, p=1.0, m=0.0):
    """(token, share, kept) of one row."""
    got = kept_of(row, T, k, p, m)
    if got is None or (T != 0 and not 0 <= u < 1):
        return -1, math.nan, -1
    order, w = got
    if T == 0:
        return int(order[0]), 1.0, 1
    mass = np.cumsum(w)
    r = min(int((mass <= float(u) * mass[-1]).sum()), len(w) - 1)
    return int(order[r]), float(w[r] / mass[-1]), len(w)


def filtered(row, T, k=0, p=1.0, m=0.0):
    """(row with -inf for what is dropped, kept)."""
    row = np.asarray(row, np.float64)
    got = kept_of(row, T, k, p, m)
    if got is None:
        return np.full(row.shape, np.nan), -1
    out = np.full(row.shape, -np.inf)
    out[got[0]] = row[got[0]]
    return out, len(got[0])
