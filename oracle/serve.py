"""Prompt attention, drafted trees, append and sampling, from their definitions in fp64 numpy.

The index sets are those of the decode step: [notes §2.1, eq. S^F / S^L], position t = place + 1.
"""
import math

import numpy as np


def _rows(q, K, V, ok):
    """o and the weighted mean of |v| for queries q [n, d] over K, V [m, d] where ok [n, m]."""
    x = np.where(ok, q @ K.T / math.sqrt(q.shape[1]), -np.inf)
    w = np.exp(x - x.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    return w @ V, w @ np.abs(V)


def prompt(q, k, v, sinks=None, window=None):
    """One sequence: q [n, Hq, d], k, v [n, Hkv, d] fp64.  Returns (o, mean |v|) [n, Hq, d]; the full
    set, or the local one where a window is given."""
    n, Hq, d = q.shape
    g = Hq // k.shape[1]
    t = np.arange(n)[:, None]
    j = np.arange(n)[None, :]
    ok = j <= t
    if window is not None:
        ok &= (j < sinks) | (j > t - window)
    o, a = np.empty_like(q), np.empty_like(q)
    for h in range(Hq):
        o[:, h], a[:, h] = _rows(q[:, h], k[:, h // g], v[:, h // g], ok)
    return o, a


def lineage(parent):
    """seen[i, j]: node j is node i or an ancestor of it."""
    n = len(parent)
    seen = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = int(parent[j])
    return seen


def tree(q, k_cache, v_cache, k_new, v_new, parent):
    """One sequence: nodes q [m, Hq, d] over the cache [n, Hkv, d] and their ancestors and themselves."""
    m, Hq, d = q.shape
    n = k_cache.shape[0]
    g = Hq // k_new.shape[1]
    ok = np.concatenate([np.ones((m, n), dtype=bool), lineage(parent)], axis=1)
    K = np.concatenate([k_cache, k_new])
    V = np.concatenate([v_cache, v_new])
    o, a = np.empty_like(q), np.empty_like(q)
    for h in range(Hq):
        o[:, h], a[:, h] = _rows(q[:, h], K[:, h // g], V[:, h // g], ok)
    return o, a


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, prob) of one row, as include/oda_serve.h defines them, in exact order and fp64 sums."""
    l = np.asarray(logits, dtype=np.float64).copy()
    l[np.isnan(l)] = -np.inf
    if not np.any(l > -np.inf):
        return -1, 0.0
    if not temperature > 0:
        return int(np.argmax(l)), 1.0
    if np.any(l == np.inf):
        l = np.where(l == np.inf, 0.0, -np.inf)
    with np.errstate(over="ignore"):
        w = np.exp((l - l.max()) / float(temperature))
    if np.isinf(temperature):
        w = np.where(l > -np.inf, 1.0, 0.0)
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -np.inf]
    if 0 < top_k < len(order):
        order = order[:top_k]
    if top_p < 1:
        mass = np.cumsum(w[order])
        n = 1 if top_p <= 0 else int(np.searchsorted(mass, float(top_p) * mass[-1])) + 1
        order = order[:max(1, n)]
    if min_p > 0:
        order = order[w[order] >= min(float(min_p), 1.0)]
    order = np.sort(order)
    mass = np.cumsum(w[order])
    uu = float(u) if u >= 0 else 0.0
    i = int(np.searchsorted(mass, min(uu, 1.0) * mass[-1], side="right"))
    i = min(i, int(np.nonzero(w[order])[0][-1]))
    return int(order[i]), float(w[order[i]] / mass[-1])


def append_places(pos, cu, rows, max_pages, n_stage, page=16):
    """[(sequence, staging row, page index of the sequence, slot)] of every appended row that is written."""
    out = []
    for b in range(len(pos)):
        for i in range(cu[b], cu[b + 1]):
            place = pos[b] - 1 + i - cu[b]
            src = i if rows is None else int(rows[i])
            if pos[b] >= 1 and place < max_pages * page and 0 <= src < n_stage:
                out.append((b, src, place // page, place % page))
    return out
