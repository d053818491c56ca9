"""The layer operators in fp64 (oracle; test infrastructure only).

Plain numpy from the operators' formulas: embedding lookup and its gradient, the
root-mean-square norm with an E4M3 output and its gradients, and the FP8
projection with its gradients.  FP8 rows carry one scale per 128 values of a row,
[groups, n]; FP8 weights one scale per 128 x 128 tile.
"""

import numpy as np

from .codecs import e4m3_decode

GROUP = 128


def spread_rows(scale, cols):
    """Scales [groups, n] of FP8 rows -> one per value, [n, cols]."""
    return np.repeat(np.asarray(scale, np.float64).T, GROUP, axis=1)[:, :cols]


def spread_tiles(scale, rows, cols):
    """Tile scales -> one per value, [rows, cols]."""
    s = np.asarray(scale, np.float64).reshape(-(-rows // GROUP), -(-cols // GROUP))
    return np.repeat(np.repeat(s, GROUP, axis=0), GROUP, axis=1)[:rows, :cols]


def decode_rows(codes, scale):
    return e4m3_decode(codes).astype(np.float64) * spread_rows(scale, codes.shape[1])


def decode_tiles(codes, scale):
    return e4m3_decode(codes).astype(np.float64) * spread_tiles(scale, *codes.shape)


def embed(table, ids, factor):
    """Rows of an fp64 table; ids outside it give zero rows."""
    out = np.zeros((len(ids), table.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < table.shape[0]:
            out[t] = factor * table[v]
    return out


def embed_grad(dy, ids, rows, factor):
    """(gradient, sum of the magnitudes of its terms)."""
    g, a = np.zeros((rows, dy.shape[1])), np.zeros((rows, dy.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < rows:
            g[v] += factor * dy[t]
            a[v] += abs(factor) * np.abs(dy[t])
    return g, a


def rmsnorm(h, weight, eps):
    """(y, rstd) of fp64 rows."""
    rstd = 1 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * weight, rstd


def rmsnorm_grad(dy, h, weight, rstd):
    """(gradient of h through the norm, gradient of the weight)."""
    u = h * rstd[:, None]
    t = dy * weight
    return rstd[:, None] * (t - u * np.mean(t * u, axis=1, keepdims=True)), np.sum(dy * u, axis=0)


def row_scales(y):
    """The scales [groups, n] of FP8 rows of y: the group's maximum magnitude / 448."""
    n, c = y.shape
    g = -(-c // GROUP)
    p = np.zeros((n, g * GROUP))
    p[:, :c] = np.abs(y)
    return (p.reshape(n, g, GROUP).max(axis=2) / 448).T
