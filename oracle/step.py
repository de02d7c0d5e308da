"""The loss over a vocabulary with its gradients (oracle; test infrastructure
only), fp64 formulas.

A row whose target is negative or past the vocabulary is left out: loss 0, no
part in the gradients, whatever it holds.
"""

import numpy as np


def counts(targets, vocab):
    t = np.asarray(targets)
    return (t >= 0) & (t < vocab)


def xent_forward(x, w, targets):
    """-> (loss, lse, logits) in fp64."""
    s = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    top = s.max(axis=1, keepdims=True)
    lse = (top + np.log(np.exp(s - top).sum(axis=1, keepdims=True)))[:, 0]
    live = counts(targets, s.shape[1])
    loss = np.zeros(len(lse))
    rows = np.flatnonzero(live)
    loss[rows] = lse[rows] - s[rows, np.asarray(targets)[rows]]
    return loss, lse, s


def xent_residual(s, lse, targets):
    """D = exp(s - lse) - [target], zero for rows left out."""
    live = counts(targets, s.shape[1])
    rows = np.flatnonzero(live)
    D = np.zeros_like(s)
    D[rows] = np.exp(s[rows] - np.asarray(lse, dtype=np.float64)[rows, None])
    D[rows, np.asarray(targets)[rows]] -= 1.0
    return D


def xent_backward(x, w, targets, lse, dloss):
    """-> (dx, dw) of sum(dloss * loss) in fp64 for the lse given."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    live = counts(targets, w.shape[0])
    x = np.where(live[:, None], x, 0.0)
    D = xent_residual(x @ w.T, lse, targets)
    g = D * np.where(live, np.asarray(dloss, dtype=np.float64), 0.0)[:, None]
    return g @ w, g.T @ x
