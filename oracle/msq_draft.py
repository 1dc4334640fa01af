"""Plain oracle of drafted tokens (numpy, fp64): sets of a tree, tree masks, verification."""
from __future__ import annotations

import numpy as np


def ancestors(parents):
    """bool [n][n]: itself and its ancestors; a parent below 0 or not smaller makes a root."""
    n = len(parents)
    sees = np.eye(n, dtype=bool)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            sees[i] |= sees[p]
    return sees


def words(sees, count):
    """uint32 [n][count] of bool [n][m]."""
    n, m = sees.shape
    bits = np.zeros((n, 32 * count), np.uint64)
    bits[:, :min(m, 32 * count)] = sees[:, :32 * count]
    return (bits.reshape(n, count, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)


def tree_sees(length, sets, window=0):
    """[n][length] which positions each of the call's rows sees: the ones before them, and of their
    own those of its set; with a window the last `window` of these."""
    n = len(sets)
    m = np.zeros((n, max(length, n)), bool)  # columns: position + max(n - length, 0)
    before = m.shape[1] - n
    m[:, :before] = length >= n
    m[:, before:] = sets
    if window:
        m &= np.cumsum(m[:, ::-1], 1)[:, ::-1] <= window
    return m[:, m.shape[1] - length:]


def _mass(row):
    row = np.asarray(row, np.float64)
    with np.errstate(invalid="ignore"):
        return np.where((row > 0) & np.isfinite(row), row, 0.0)


def _number(u):
    return min(float(u), 1.0) if u > 0 else 0.0


def verify(tokens, parents, target, draft=None, uniform=None):
    """One sequence: (next token, rows kept).  parents None: a chain."""
    n, V = len(tokens), target.shape[1]
    parents = [i - 1 if parents is None else int(parents[i]) for i in range(n)]
    if n == 0:
        return -1, []
    children = {i: [j for j in range(1, n) if parents[j] == i and i < j] for i in range(n)}
    at, path = 0, [0]
    if uniform is None:
        while True:
            row = np.asarray(target[at], np.float64)
            best = -1 if np.isnan(row).all() else int(np.nanargmax(row))
            hit = [j for j in children[at] if tokens[j] == best]
            if best < 0 or not hit:
                return best, path
            at = hit[0]
            path.append(at)
    while True:
        start = _mass(target[at])
        r, m = start.copy(), 1.0
        for j in children[at]:
            x = int(tokens[j])
            inside = 0 <= x < V
            rx = r[x] if inside else 0.0
            q = _mass(draft[at]) if draft is not None else None
            qx = (q[x] if inside else 0.0) if draft is not None else 1.0
            if inside and _number(uniform[j]) * qx * m < rx:
                at = j
                path.append(j)
                break
            if draft is not None:
                r = np.maximum(r / (m if m > 0 else 1.0) - q, 0.0)
                m = r.sum()
            else:
                m -= rx
                if inside:
                    r[x] = 0.0
        else:
            if not r.sum() > 0:
                r = start
            run = np.cumsum(r)
            if not run[-1] > 0:
                return -1, path
            t = int(np.searchsorted(run, _number(uniform[0]) * run[-1], side="right"))
            return min(t, int(np.flatnonzero(r)[-1])), path
