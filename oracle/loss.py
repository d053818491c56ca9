"""The softmax losses over an FP8 head in fp64 (oracle; test infrastructure only).

Plain numpy from the formulas.  x [n, cols] and w [rows, cols] are the decoded FP8 rows and
weight; targets are pairs (ids [n, k], weights [n, k]), a pair with weight 0 saying
nothing; a row without a pair that counts has loss 0 and no gradient.
"""

import numpy as np


def class_pairs(targets, rows):
    """(ids, weights, which count) of one class a row."""
    ids = np.asarray(targets, np.int64)[:, None]
    kept = (ids >= 0) & (ids < rows)
    return np.where(kept, ids, 0), kept.astype(np.float64), kept


def teacher_pairs(ids, logits, scale, rows):
    """The same of a teacher's top logits: the softmax over the pairs that count."""
    ids, z = np.asarray(ids, np.int64), np.asarray(logits, np.float64)
    kept = (ids >= 0) & (ids < rows) & ~np.isneginf(z)
    z = scale * np.where(kept, z, 0)
    top = np.max(np.where(kept, z, -np.inf), axis=1, keepdims=True)
    e = np.where(kept, np.exp(np.where(kept, z - np.where(np.isfinite(top), top, 0), 0)), 0)
    total = e.sum(axis=1, keepdims=True)
    return np.where(kept, ids, 0), e / np.where(total > 0, total, 1), kept


def logits(x, w, scale):
    """(z, sum of the magnitudes of its terms)."""
    return scale * (x @ w.T), abs(scale) * (np.abs(x) @ np.abs(w).T)


def log_sum(z):
    """log sum exp of rows."""
    top = z.max(axis=1, keepdims=True)
    return (top + np.log(np.exp(z - top).sum(axis=1, keepdims=True)))[:, 0]


def log_probs(z, ids):
    """z[t, ids[t, i]] - log_sum(z)[t], exact for probabilities near 1 too: the largest logit stays out of the
    sum of exponentials."""
    best = z.argmax(axis=1)[:, None]
    behind = z - np.take_along_axis(z, best, 1)
    others = np.exp(behind)
    np.put_along_axis(others, best, 0.0, 1)
    return np.take_along_axis(behind, ids, 1) - np.log1p(others.sum(axis=1, keepdims=True))


def loss(z, pairs):
    """(loss, log-sum, log-probabilities with 0 for pairs that do not count)."""
    ids, q, kept = pairs
    logp = np.where(kept, log_probs(z, ids), 0.0)
    terms = np.where(q > 0, q * (np.log(np.where(q > 0, q, 1)) - logp), 0.0)
    return terms.sum(axis=1), log_sum(z), logp


def weights_of(pairs, rows):
    """The targets' weights as a matrix [n, rows]."""
    ids, q, _ = pairs
    out = np.zeros((ids.shape[0], rows))
    np.add.at(out, (np.arange(ids.shape[0])[:, None], ids), q)
    return out


def dlogits(z, pairs):
    """The gradient of each row's loss to its logits z."""
    p = np.exp(z - log_sum(z)[:, None])
    return np.where(pairs[2].any(axis=1)[:, None], p - weights_of(pairs, z.shape[1]), 0.0)


def grads(x, w, z, pairs, dloss, scale):
    """(dx, dw) and the sums of their terms' magnitudes."""
    u = dlogits(z, pairs) * np.where(pairs[2].any(axis=1), scale * np.asarray(dloss, np.float64), 0.0)[:, None]
    return u @ w, u.T @ x, np.abs(u) @ np.abs(w), np.abs(u).T @ np.abs(x)
