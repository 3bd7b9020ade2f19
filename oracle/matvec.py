"""A few rows times one 4-bit matrix with group scales, in 64 bits.

y[t, n] = bias[n] + sum_k W[n, k] x[t, k] with W[n, k] = s[n, g(k)] * (v(code) - z[n, g(k)]).
Pinned by ``tests/test_oracle_operators.py`` against the stacks' own dequantisers and a
scalar loop.
"""

from __future__ import annotations

import numpy as np

from .mxfp4 import e2m1_value, e8m0_value, unpack_mx
from .nf4 import codebook, unpack_codes


def matvec_weight(codes, scales, quant_type: str, group: int, zeros=None) -> np.ndarray:
    """The matrix [N, K] in fp64 (``scales`` as values; e8m0 bytes for mxfp4)."""
    N = codes.shape[0]
    if quant_type == "mxfp4":
        v = e2m1_value(unpack_mx(codes)).astype(np.float64)
        s = e8m0_value(scales).astype(np.float64)
    else:
        c = unpack_codes(codes)
        v = c.astype(np.float64) if quant_type == "int4" else \
            codebook(quant_type).astype(np.float64)[c]
        s = np.asarray(scales, dtype=np.float64)
    v = v.reshape(N, -1, group)
    if quant_type == "int4":
        z = np.full(s.shape, 8.0) if zeros is None else zeros.astype(np.float64)
        v = v - z[:, :, None]
    return (v * s[:, :, None]).reshape(N, -1)


def matvec(x, codes, scales, quant_type: str, group: int, zeros=None, bias=None):
    """(y, sum_k |W x| + |bias|), both [T, N] fp64."""
    w = matvec_weight(codes, scales, quant_type, group, zeros)
    x = np.asarray(x, dtype=np.float64)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, mag = y + bias.astype(np.float64), mag + np.abs(bias)
    return y, mag
