"""Dispatch of rows to experts and back, its gradients, and the router's
gradient -- oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Sources.  "mxfp6-sm120" page, section "Execution model" (indirect routing: rows
are gathered per expert through an index list; the reduction that brings them
back), and "TokenSpeed SiTU" page, section "Supported contract" (each rank
keeps only the experts of its contiguous shard).  The gradients are the plain
derivatives of these definitions.

Every function walks tokens and slots one by one, in float64.
"""
from __future__ import annotations

import numpy as np


def row_of(ids: np.ndarray, num_experts: int, local_offset: int = 0, local_count: int | None = None) -> np.ndarray:
    """[T, k] row of each assignment when the local assignments are ordered by
    (expert, token), -1 for experts outside the shard."""
    if local_count is None:
        local_count = num_experts
    T, k = ids.shape
    out = np.full((T, k), -1, dtype=np.int64)
    p = 0
    for e in range(local_offset, local_offset + local_count):
        for t in range(T):
            for j in range(k):
                if ids[t, j] == e:
                    out[t, j] = p
                    p += 1
    return out


def permute(x: np.ndarray, rows_of: np.ndarray, rows: np.ndarray) -> np.ndarray:
    """rows with row p replaced by the token row it belongs to."""
    out = rows.copy()
    for t, j in zip(*np.nonzero(rows_of >= 0)):
        out[rows_of[t, j]] = x[t]
    return out


def unpermute(rows: np.ndarray, rows_of: np.ndarray, w: np.ndarray | None = None, residual: np.ndarray | None = None):
    """(y, sum of the magnitudes added up in each element of y)."""
    T, k = rows_of.shape
    y = np.zeros((T, rows.shape[1])) if residual is None else residual.astype(np.float64)
    size = np.abs(y)
    for t in range(T):
        for j in range(k):
            if rows_of[t, j] >= 0:
                term = rows[rows_of[t, j]] * (1.0 if w is None else w[t, j])
                y[t] += term
                size[t] += np.abs(term)
    return y, size


def unpermute_backward(dy: np.ndarray, rows: np.ndarray, rows_of: np.ndarray, w: np.ndarray, drows: np.ndarray):
    """(drows with the named rows replaced, dw, sum of magnitudes in each dw)."""
    out, dw, size = drows.copy(), np.zeros(w.shape), np.zeros(w.shape)
    for t, j in zip(*np.nonzero(rows_of >= 0)):
        p = rows_of[t, j]
        out[p] = w[t, j] * dy[t]
        dw[t, j] = np.sum(dy[t] * rows[p])
        size[t, j] = np.sum(np.abs(dy[t] * rows[p]))
    return out, dw, size


def route_backward(ids: np.ndarray, w: np.ndarray, dw: np.ndarray, num_experts: int) -> np.ndarray:
    """dlogits [T, E] through the softmax over each token's chosen logits."""
    T, k = ids.shape
    out = np.zeros((T, num_experts))
    for t in range(T):
        jac = np.diag(w[t]) - np.outer(w[t], w[t])
        out[t, ids[t]] = jac @ dw[t]
    return out
