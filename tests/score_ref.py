"""The operators around the search, from their definitions in 64 bits (numpy)."""

import numpy as np


def unpack(weights, K):
    """q [N, K] of packed weights [N, ceil(K / 2)]."""
    q = np.empty((weights.shape[0], 2 * weights.shape[1]), np.int64)
    q[:, 0::2] = weights & 15
    q[:, 1::2] = weights >> 4
    return q[:, :K]


def layer(x, weights, scales, zeros, bias, K, group):
    """(y, sum of the absolute terms) of hidden states x [M, K]."""
    q = unpack(weights, K)
    g = np.arange(K) // group
    z = 8 if zeros is None else (zeros & 15).astype(np.int64)[:, g]
    w = (q - z) * scales.astype(np.float64)[:, g]
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        y = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    if bias is not None:
        y = y + bias
        size = size + np.abs(bias)
    return y, size


def log_softmax(x, scale=1.0, bias=None):
    z = x.astype(np.float64) * scale
    if bias is not None:
        z = z + bias
    out = np.empty_like(z)
    for r, row in enumerate(z):
        if np.isnan(row).any() or (row == np.inf).any():
            out[r] = np.nan
        elif (row == -np.inf).all():
            out[r] = -np.inf
        else:
            d = row - row.max()
            e = np.exp(d)
            e[np.argmax(d)] = 0.0                 # one of the largest: exactly 1, left to log1p
            out[r] = d - np.log1p(e.sum())
    return out


def sample_row(x, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log-probability, kept) of one row."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    T, top_p, min_p, u = (float(np.float32(v)) for v in (T, top_p, min_p, u))
    valid = np.flatnonzero(x > -np.inf)
    if valid.size == 0:
        return -1, -np.inf, 0
    m = x.max()
    if m == np.inf:
        valid = np.flatnonzero(x == np.inf)
    if not T > 0:
        return int(np.flatnonzero(x == m)[0]), 0.0, 1
    order = valid[np.argsort(-x[valid], kind="stable")]
    mass = np.ones(order.size) if m == np.inf else np.exp((x[order] - m) / T)
    if top_k > 0:
        order, mass = order[:top_k], mass[:top_k]
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(mass)[:-1]))
        n = max(1, int((before < top_p * mass.sum()).sum()))
        order, mass = order[:n], mass[:n]
    if min_p > 0:
        ok = mass >= min(min_p, 1.0)
        order, mass = order[ok], mass[ok]
    back = np.argsort(order)
    order, mass = order[back], mass[back]
    run = np.cumsum(mass)
    u = min(max(u, 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
    i = int(np.argmax(run > u * run[-1]))
    return int(order[i]), float(np.log(mass[i] / run[-1])), order.size


def sample(x, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    R = x.shape[0]
    rows = [np.broadcast_to(np.asarray(v), (R,)) for v in (T, top_k, top_p, min_p)]
    res = [sample_row(x[r], u[r], *(v[r] for v in rows)) for r in range(R)]
    return (np.array([r[0] for r in res], np.int64), np.array([r[1] for r in res]),
            np.array([r[2] for r in res], np.int64))
