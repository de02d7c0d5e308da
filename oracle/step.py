"""The loss over a vocabulary and the norms between blocks, with their gradients,
and gradient clipping (oracle; test infrastructure only), fp64 formulas.

A row whose target is negative or past the vocabulary is left out: loss 0, no
part in the gradients, whatever it holds.
"""

import numpy as np

from . import layer as ol


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


def _gates(gate, rows, d):
    """The gate of every row."""
    if gate is None:
        return np.ones((rows, d))
    gate = np.asarray(gate, dtype=np.float64).reshape(-1, d)
    return np.repeat(gate, rows // gate.shape[0], axis=0)


def block_norm_forward(y, h, weight=None, bias=None, eps=1e-5, post=True, post_weight=None, post_bias=None, gate=None,
                       scale=1.0, layer=False):
    """-> (x, h', stats (4 x rows)) in fp64."""
    y, h = np.asarray(y, dtype=np.float64), np.asarray(h, dtype=np.float64)
    rows, d = y.shape
    n, pm, pr = y, np.zeros(rows), np.ones(rows)
    if post:
        n, pm, pr = ol.norm_forward(y, post_weight, post_bias, eps, layer)
    h2 = scale * h + _gates(gate, rows, d) * n
    x, m, r = ol.norm_forward(h2, weight, bias, eps, layer)
    return x, h2, np.stack([pm, pr, m, r])


def block_norm_backward(dx, dh, y, h2, stats, weight=None, post=True, post_weight=None, post_bias=None, gate=None,
                        scale=1.0, layer=False):
    """-> dict of the gradients in fp64 for the statistics given."""
    y = np.asarray(y, dtype=np.float64)
    rows, d = y.shape
    pm, pr, m, r = np.asarray(stats, dtype=np.float64)
    t, dweight, dbias = ol.norm_backward(dx, h2, weight, m, r, layer)
    if dh is not None:
        t = t + np.asarray(dh, dtype=np.float64)
    k = _gates(gate, rows, d)
    out = {"dh": scale * t, "dweight": dweight, "dbias": dbias, "t": t}
    n = y
    if post:
        n = (y - (pm[:, None] if layer else 0.0)) * pr[:, None]
        out["dy"], out["dpost_weight"], out["dpost_bias"] = ol.norm_backward(k * t, y, post_weight, pm, pr, layer)
        if post_weight is not None:
            n = n * post_weight
        if post_bias is not None:
            n = n + post_bias
    else:
        out["dy"] = k * t
    groups = 1 if gate is None else np.asarray(gate).size // d
    out["dgate"] = (t * n).reshape(groups, rows // groups, d).sum(axis=1)
    return out


def grad_clip(tensors, max_norm=None, eps=1e-6, sumsq=None):
    """-> (sum of squares, norm, clipped tensors) in fp64."""
    tensors = [np.asarray(t, dtype=np.float64) for t in tensors]
    q = sum((t * t).sum() for t in tensors) if sumsq is None else sumsq
    norm = np.sqrt(q)
    c = 1.0 if max_norm is None or q == 0 else min(1.0, max_norm / (norm + eps))
    return q, norm, [t * c for t in tensors]
