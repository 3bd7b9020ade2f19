"""RMS norms after and before a block with its gate and residual scale, and
their gradients, in 64 bits:

    z = y * rstd(y) * w_post,  r = beta * residual + alpha * gate * z,
    h = r * rstd(r) * w_pre,   rstd(v) = (mean(v^2) + eps)^(-1/2).

Weights are given with their offset already added; ``gate`` broadcasts to [T, H].
Every function also returns the size of the terms it adds (the same sums over
absolute values), which bounds the rounding of a 32-bit evaluation.
Pinned by ``tests/test_oracle_operators.py`` against differences.
"""

from __future__ import annotations

import numpy as np


def _f8(v):
    return np.asarray(v, dtype=np.float64)


def rstd(v, eps):
    return 1.0 / np.sqrt(np.mean(_f8(v) ** 2, axis=1, keepdims=True) + eps)


def post(residual, y, w_post, gate, alpha, beta, eps):
    """(r, its terms' size); ``w_post`` None: y as it is."""
    z = _f8(y)
    if w_post is not None:
        z = z * rstd(y, eps) * _f8(w_post)
    a, b = beta * _f8(residual), alpha * _f8(gate) * z
    return a + b, np.abs(a) + np.abs(b)


def pre(r, w_pre, eps):
    return _f8(r) * rstd(r, eps) * _f8(w_pre)


def rms_grad(g, x, w, eps):
    """Gradient of x * rstd(x) * w: (dx, its terms' size, dw per row)."""
    g, x, w = _f8(g), _f8(x), _f8(w)
    s = rstd(x, eps)
    a, b = s * g * w, x * s ** 3 * np.mean(g * w * x, axis=1, keepdims=True)
    size = np.abs(a) + np.abs(x) * s ** 3 * np.mean(np.abs(g * w * x), axis=1, keepdims=True)
    return a - b, size, g * x * s


def backward(dh, d_r, r, y, w_pre, w_post, gate, alpha, beta, eps):
    """Gradients and sizes: dict name -> (value, size); ``gate`` [T, 1], [1, H] or 1."""
    out = {}
    dr, size = 0.0 * _f8(r), 0.0 * _f8(r)
    if d_r is not None:
        dr, size = dr + _f8(d_r), size + np.abs(_f8(d_r))
    if dh is not None:
        d, sz, dw = rms_grad(dh, r, w_pre, eps)
        dr, size = dr + d, size + sz
        out["dw_pre"] = (dw.sum(0), np.abs(dw).sum(0))
    out["dresidual"] = (beta * dr, abs(beta) * size)
    if y is None:
        return out
    gate = _f8(gate)
    z = _f8(y)
    if w_post is not None:
        z = z * rstd(y, eps) * _f8(w_post)
    if gate.ndim == 2:
        axis = 1 if gate.shape[1] == 1 else 0
        out["dgate"] = (alpha * (dr * z).sum(axis), abs(alpha) * (size * np.abs(z)).sum(axis))
    dz, dzs = alpha * gate * dr, np.abs(alpha * gate) * size
    if w_post is None:
        out["dy"] = (dz, dzs)
        return out
    dy, _, dw = rms_grad(dz, y, w_post, eps)
    out["dy"] = (dy, rms_grad(dzs, np.abs(_f8(y)), np.abs(_f8(w_post)), eps)[1])
    out["dw_post"] = (dw.sum(0), (dzs * np.abs(_f8(y)) * rstd(y, eps)).sum(0))
    return out
