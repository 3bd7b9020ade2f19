"""Newton-Schulz orthogonalisation of per-expert factors and the optimiser step
around it, in 64 bits.

X_0 = u / (|u|_F + eps); X <- a X + b (X X^T) X + c (X X^T)^2 X per step.
Pinned by ``tests/test_oracle_operators.py`` against the same polynomial of the
singular values.
"""

from __future__ import annotations

import numpy as np


def newton_schulz(u, steps: int, coeffs, eps: float) -> np.ndarray:
    """u [E, m, n]; the products go through the shorter side."""
    a, b, c = coeffs
    x = np.asarray(u, dtype=np.float64)
    wide = x.shape[1] <= x.shape[2]
    x = x if wide else x.transpose(0, 2, 1)
    x = x / (np.sqrt((x ** 2).sum(axis=(1, 2), keepdims=True)) + eps) if eps > 0 or x.any() else x
    for _ in range(steps):
        g = x @ x.transpose(0, 2, 1)
        x = a * x + (b * g + c * (g @ g)) @ x
    return x if wide else x.transpose(0, 2, 1)


def muon_momentum(grad, m, mu):
    return mu * np.asarray(m, np.float64) + np.asarray(grad, np.float64)


def muon_weight(w, o, lr, weight_decay, scale):
    return np.asarray(w, np.float64) * (1.0 - lr * weight_decay) - lr * scale * o
