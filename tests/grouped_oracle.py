"""The grouped products in 64 bits, from their definition (numpy only, no code
of the library)."""
import numpy as np


def edges(offsets, T):
    """(start, end) of every group's rows: offsets within 0 .. T, none below
    an earlier one."""
    o = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, T))
    return list(zip(o[:-1], o[1:]))


def outside(offsets, T):
    """Which rows belong to no group."""
    free = np.ones(T, bool)
    for a, b in edges(offsets, T):
        free[a:b] = False
    return free


def product(x, w, offsets):
    """(y, sum of magnitudes), zero rows where there is no group; w groups x K
    x N."""
    T, N = x.shape[0], w.shape[2]
    y, size = np.zeros((T, N)), np.zeros((T, N))
    for g, (a, b) in enumerate(edges(offsets, T)):
        y[a:b] = x[a:b] @ w[g]
        size[a:b] = np.abs(x[a:b]) @ np.abs(w[g])
    return y, size


def gradient(x, dy, offsets):
    """(dw, sum of magnitudes), groups x K x N."""
    rows = edges(offsets, x.shape[0])
    dw, size = np.zeros((2, len(rows), x.shape[1], dy.shape[1]))
    for g, (a, b) in enumerate(rows):
        dw[g] = x[a:b].T @ dy[a:b]
        size[g] = np.abs(x[a:b]).T @ np.abs(dy[a:b])
    return dw, size
