"""Adapters beside the output layer and scores of given tokens, from their definitions in 64 bits (numpy)."""

import numpy as np


def adapters(x, ids, slots):
    """(sum, sum of the absolute terms) that the adapters add for rows x [M, K]; slots: {id: (down, up, scale)}."""
    x = x.astype(np.float64)
    N = next(iter(slots.values()))[1].shape[0] if slots else 0
    y, size = np.zeros((x.shape[0], N)), np.zeros((x.shape[0], N))
    for m, i in enumerate(ids):
        if int(i) not in slots:
            continue
        down, up, scale = (np.asarray(v, np.float64) for v in slots[int(i)])
        with np.errstate(invalid="ignore"):
            y[m] = up @ (scale * (down @ x[m]))
        size[m] = np.abs(up) @ (np.abs(scale) * (np.abs(down) @ np.abs(x[m])))
    return y, size


def _order(x):
    """Labels from the largest score to the smallest, ties to the lowest index, NaN as -inf."""
    return np.argsort(-np.where(np.isnan(x), -np.inf, x), kind="stable")


def scores_row(x, tokens, n, T=1.0):
    """(log-probabilities, ranks, entropy, top tokens, top log-probabilities) of one row."""
    x = x.astype(np.float64)
    V = x.size
    T = float(np.float32(T))
    T = min(T, float(np.finfo(np.float32).max)) if T > 0 else 0.0
    order = _order(x)
    place = np.empty(V, np.int64)
    place[order] = np.arange(V)
    valid = x > -np.inf
    if np.isnan(x).any() or (x == np.inf).any():
        lp, ent = np.full(V, np.nan), np.nan
    elif not valid.any():
        lp, ent = np.full(V, -np.inf), 0.0
    elif T == 0.0:
        lp, ent = np.full(V, -np.inf), 0.0
        lp[order[0]] = 0.0
    else:
        with np.errstate(over="ignore", under="ignore"):
            d = (x - x.max()) / T
            e = np.exp(d)
            e[order[0]] = 0.0                        # one of the largest: exactly 1, left to log1p
            lz = np.log1p(e.sum())
            ent = lz + (np.where(e > 0, -d, 0.0) * e).sum() / (1.0 + e.sum())
            lp = d - lz
    ok = (tokens >= 0) & (tokens < V)
    at = np.where(ok, tokens, 0)
    top = order[:n]
    listed = valid[top]
    pad = n - top.size
    tt = np.concatenate((np.where(listed, top, -1), np.full(pad, -1)))
    tl = np.concatenate((np.where(listed, lp[top], -np.inf), np.full(pad, -np.inf)))
    return np.where(ok, lp[at], -np.inf), np.where(ok, place[at], -1), ent, tt, tl


def scores(x, tokens, n, T=1.0):
    R = x.shape[0]
    Ts = np.broadcast_to(np.asarray(T), (R,))
    rows = [scores_row(x[r], tokens[r], n, Ts[r]) for r in range(R)]
    return tuple(np.array([r[i] for r in rows]) for i in range(5))
