"""Token rows into expert rows and back, in 64 bits -- oracle.

TEST INFRASTRUCTURE ONLY -- see ``oracle/__init__.py``.

Pair p = t*k + j has its row at ``pos[p]``; one outside [0, R) has none.  Pinned by
``tests/test_oracle_dispatch.py`` against the layer's own sum and against differences.
"""

from __future__ import annotations

import numpy as np


def _pairs(pos, k, R):
    pos = np.asarray(pos, dtype=np.int64).reshape(-1)
    p = np.flatnonzero((pos >= 0) & (pos < R))
    return p, p // k, pos[p]


def _weights(w, n):
    return np.ones(n) if w is None else np.asarray(w, dtype=np.float64).reshape(-1)


def dispatch(x, pos, k, rows, w=None):
    """``rows`` [R, H] with the named ones replaced."""
    out = np.array(rows, dtype=np.float64)
    p, t, at = _pairs(pos, k, len(out))
    out[at] = _weights(w, np.size(pos))[p, None] * np.asarray(x, np.float64)[t]
    return out


def combine(rows, pos, k, w=None):
    rows = np.asarray(rows, dtype=np.float64)
    p, t, at = _pairs(pos, k, len(rows))
    y = np.zeros((np.size(pos) // k, rows.shape[1]))
    np.add.at(y, t, _weights(w, np.size(pos))[p, None] * rows[at])
    return y


def combine_backward(dy, rows, pos, k, w=None):
    """(drows, zero where no pair is; dw [T, k])."""
    dy, rows = np.asarray(dy, np.float64), np.asarray(rows, np.float64)
    p, t, at = _pairs(pos, k, len(rows))
    dw = np.zeros(np.size(pos))
    dw[p] = (dy[t] * rows[at]).sum(1)
    return dispatch(dy, pos, k, np.zeros_like(rows), w), dw.reshape(-1, k)


def route_weights(logits, ids, renormalize=True):
    z = np.asarray(logits, np.float64)
    ids = np.asarray(ids, np.int64)
    z = np.exp(z - z.max(1, keepdims=True))
    w = np.take_along_axis(z, ids, 1)
    return w / (w if renormalize else z).sum(1, keepdims=True)


def route_backward(logits, ids, dw, renormalize=True):
    """dL/dlogits [T, E] from dL/dw [T, k] by the softmax's own Jacobian."""
    ids, dw = np.asarray(ids, np.int64), np.asarray(dw, np.float64)
    E = np.shape(logits)[1]
    w = route_weights(logits, ids, renormalize)
    out = np.zeros((len(ids), E))
    for t in range(len(ids)):
        pick = np.eye(E)[ids[t]]  # [k, E]
        if renormalize:
            jac = np.diag(w[t]) - np.outer(w[t], w[t])  # dw_i / dlogit of the j-th chosen
            out[t] = dw[t] @ jac @ pick
        else:
            p = route_weights(logits[t:t + 1], np.arange(E)[None], False)[0]
            out[t] = dw[t] @ (w[t][:, None] * (pick - p))
    return out
