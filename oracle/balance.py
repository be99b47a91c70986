"""Balance of the router: load-balance loss, z-loss, tokens per expert, and the
gradient of both losses -- oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Sources.  "TokenSpeed SiTU" page, section "Supported contract" (global top-k ids over
all experts); the pages train nothing, so the losses are the plain ones: per
sequence E sum_e f_e P_e, f_e the share of the assignments that went to expert e
and P_e the mean of its softmax probability, averaged over the sequences; and the
mean of the squared log-sum-exp.  The counts are constants for the gradient.

Everything walks token by token, in float64.  Next to each result stands the sum
that bounds fp32's error on it: an exponential is off by its argument's rounding
(|x - max| half steps) and a few more, so a probability p carries p (|x - max| + c)
half steps of fp32, and sums of them add up.
"""
from __future__ import annotations

import numpy as np


def counted(logits: np.ndarray, offsets, mask=None) -> np.ndarray:
    """Sequence of each token, -1 for one that does not count."""
    T = logits.shape[0]
    seq = np.full(T, -1)
    for s in range(len(offsets) - 1):
        for t in range(max(offsets[s], 0), min(offsets[s + 1], T)):
            if (mask is None or mask[t]) and np.any(logits[t] != -np.inf):
                seq[t] = s
    return seq


def _softmax(x: np.ndarray):
    """(p, log-sum-exp, |x - max| where p is not 0) of one token."""
    m = np.max(x)
    e = np.exp(x - m)
    s = np.sum(e)
    return e / s, m + np.log(s), np.where(e > 0, np.abs(x - m), 0.0)


def balance(logits, ids, num_seqs: int, offsets, mask=None):
    """(losses [2], counts [S, E], tokens [S + 2], lse [T], and the sums that bound
    the error of the losses [2] and of lse [T] in units of fp32's half step)."""
    T, E = logits.shape
    k = ids.shape[1]
    seq = counted(logits, offsets, mask)
    counts = np.zeros((num_seqs, E), dtype=np.int64)
    probs, psize = np.zeros((num_seqs, E)), np.zeros((num_seqs, E))
    n = np.zeros(num_seqs, dtype=np.int64)
    lse, lsize = np.full(T, -np.inf), np.zeros(T)
    z = zsize = 0.0
    for t in range(T):
        s = seq[t]
        if s < 0:
            continue
        p, lse[t], d = _softmax(logits[t])
        rel = np.sum(p * (d + 28))  # of the sum of exponentials
        lsize[t] = rel + 2 * abs(lse[t]) + 2 * np.log(E)
        n[s] += 1
        probs[s] += p
        psize[s] += p * (d + rel + 80)
        z += lse[t] ** 2
        zsize += 2 * abs(lse[t]) * lsize[t] + 64 * lse[t] ** 2
        for e in ids[t]:
            if 0 <= e < E:
                counts[s, e] += 1
    total, used = int(n.sum()), int((n > 0).sum())
    loss, size = np.zeros(2), np.zeros(2)
    for s in range(num_seqs):
        if n[s]:
            f = counts[s] / (k * n[s])
            loss[0] += E * np.sum(f * probs[s] / n[s]) / used
            size[0] += E * np.sum(f * psize[s] / n[s]) / used
    if total:
        loss[1], size[1] = z / total, zsize / total
    return loss, counts, np.concatenate([n, [total, used]]), lse, size + 2 * np.abs(loss), lsize


def balance_backward(dloss, logits, counts, tokens, k: int, offsets, mask=None, add=None):
    """(dlogits [T, E], the sum that bounds its error in units of fp32's half step)."""
    T, E = logits.shape
    seq = counted(logits, offsets, mask)
    total, used = tokens[-2], tokens[-1]
    out = np.zeros((T, E)) if add is None else add.astype(np.float64).copy()
    size = np.zeros((T, E))
    for t in range(T):
        s = seq[t]
        if s < 0:
            continue
        p, lse, d = _softmax(logits[t])
        f = counts[s] / (k * tokens[s])
        rel = np.where(p > 0, np.abs(logits[t] - lse) + np.sum(p * (d + 28)) + 2 * abs(lse) + 2 * np.log(E) + 8, 0.0)
        dot = np.sum(f * p)
        dot_size = np.sum(f * p * (rel + 24))
        a, b = dloss[0] * E / (used * tokens[s]), dloss[1] * 2 / total
        out[t] += a * p * (f - dot) + b * lse * p
        size[t] += abs(a) * p * ((rel + 8) * (f + dot) + dot_size)
        size[t] += abs(b) * p * (abs(lse) * (rel + 8) + np.sum(p * (d + 28)) + 2 * abs(lse) + 2 * np.log(E))
    return out, size + 2 * np.abs(out)
