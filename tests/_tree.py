"""Trees of drafted tokens for the tests: topologies, and what the definitions give for them in float64 (numpy, from
the oracle's sequential functions applied along each node's path)."""
from __future__ import annotations

import numpy as np

from oracle import csa_oracle as O
from tests._common import f64

NONE = -2


def chain(T):
    return [i - 1 for i in range(T)]


def star(T):
    return [-1] * T


def binary(T):
    return [(i - 1) // 2 if i else -1 for i in range(T)]


def bushy(T, seed=0):
    """Mostly children of recent nodes, a few of any earlier node or of the last committed token."""
    r = np.random.default_rng([11, seed, T])
    return [-1 if i == 0 else int(r.integers(max(0, i - 5), i)) if r.random() < 0.8 else int(r.integers(-1, i))
            for i in range(T)]


def padded(par, T):
    return list(par) + [NONE] * (T - len(par))


def paths(par):
    """Each node's path from its root (None: an unused slot)."""
    out = []
    for i, p in enumerate(par):
        out.append(None if p < -1 else [i] if p == -1 else out[p] + [i])
    return out


def norm_rope(x, weight, norm, eps, p, inv_freq):
    """x [heads, dim] of one token at position p, in float64 (inv_freq None: no rotation)."""
    y = f64(x)
    if norm:
        y = O.rms_norm(y, np.ones(y.shape[-1]) if weight is None else f64(weight), eps)
    return y if inv_freq is None else O.rope(y, p, inv_freq)


def columns(layer, path, p0, T):
    """The score columns that a node sees: committed rows, then those of the path's nodes that complete a window."""
    n = p0 // layer.ratio
    return list(range(n)) + [n + a for k, a in enumerate(path) if (p0 + k + 1) % layer.ratio == 0]


def scores_row(layer, iq, iw, ikeys, rows_i, path, p0):
    """A node's scores over n + T columns (rotated iq), and the same with every product taken absolutely."""
    n, T = p0 // layer.ratio, len(rows_i)
    keys = np.concatenate([f64(ikeys)[:n], f64(rows_i)])
    w = f64(iw) * (layer.Di ** -0.5) * (layer.Hi ** -0.5)
    s = (w[:, None] * np.maximum(f64(iq) @ keys.T, 0.0)).sum(0)
    bound = (np.abs(w)[:, None] * (np.abs(f64(iq)) @ np.abs(keys).T)).sum(0)
    seen = np.zeros(n + T, dtype=bool)
    seen[columns(layer, path, p0, T)] = True
    return np.where(seen, s, -np.inf), np.where(seen, bound, 0.0)


def select(layer, scores, path, p0, T):
    """The selected columns, ascending (scores None: every visible one)."""
    cols = np.array(columns(layer, path, p0, T), dtype=np.int64)
    if scores is None or len(cols) <= layer.topk:
        return cols
    v = np.asarray(scores, dtype=np.float64)[cols]
    v = np.where(v == 0, 0.0, v)  # -0 and +0 tie
    order = sorted(range(len(cols)), key=lambda k: (-v[k], k))
    return cols[sorted(order[:layer.topk])]


def keys(layer, q, kv, sink, window, pool, rows_a, cols, path, p0, inv_freq):
    """The rows that a node attends to, in float64 [keys, D] (arguments as output's)."""
    n = p0 // layer.ratio
    p = p0 + len(path) - 1
    Wr = window.shape[0]
    rows = [f64(pool[c]) if c < n else f64(rows_a[c - n]) for c in cols]
    rows += [f64(window[t % Wr]) if t < p0 else f64(kv[path[t - p0]]) for t in O.window_tokens(layer, p)]
    return np.stack(rows)


def output(layer, q, kv, sink, window, pool, rows_a, cols, path, p0, inv_freq):
    """A node's attention output in float64 (rotated q)."""
    k = keys(layer, q, kv, sink, window, pool, rows_a, cols, path, p0, inv_freq)
    return O.rope(O.attend(layer, f64(q), k, sink), p0 + len(path) - 1, inv_freq, inverse=True)
