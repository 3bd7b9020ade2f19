"""Pins of the oracle's MXFP4 quantiser, product and dispatch (CPU only)."""

import numpy as np
import pytest

import oracle
from oracle import dispatch


def test_quantiser_on_values_by_hand():
    # largest 6: e = 0; ties 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    x = np.zeros(32)
    x[:12] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5.001, 7.9, -0.0, -0.2500001]
    b, s = oracle.quantize_mxfp4(x)
    assert s.tolist() == [127]
    assert oracle.unpack_mx(b)[:12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 15, 7, 8, 9]


@pytest.mark.parametrize("top,byte", [(4.0, 127), (7.99, 127), (8.0, 128), (3.99, 126), (0.0, 0),
                                      (2.0 ** -149, 0), (2.0 ** -125, 0), (2.0 ** -124, 1),
                                      (3.4e38, 252)])
def test_scale_bytes(top, byte):
    x = np.zeros((1, 32))
    x[0, 5] = -top
    b, s = oracle.quantize_mxfp4(x)
    assert s[0, 0] == byte
    assert abs(oracle.dequantize_mxfp4(b, s)[0, 5] + top) <= max(0.25 * top, 2.0 ** -129)


def test_non_finite_blocks():
    x = np.ones((1, 96))
    x[0, 3], x[0, 40] = np.inf, np.nan
    b, s = oracle.quantize_mxfp4(x)
    v = oracle.dequantize_mxfp4(b, s)
    assert np.isnan(v[0, :64]).all() and (v[0, 64:] == 1).all()


def test_what_blocks_stand_for_is_quantised_to_itself():
    # a block's largest is rounded to 4 or 6 of its scale, so the scale stays
    x = np.random.default_rng(0).standard_normal((40, 64)) * 2.0 ** np.arange(-20, 20)[:, None]
    b, s = oracle.quantize_mxfp4(x)
    b2, s2 = oracle.quantize_mxfp4(oracle.dequantize_mxfp4(b, s))
    assert np.array_equal(b, b2) and np.array_equal(s, s2)


def test_product_is_the_sum_over_blocks():
    rng = np.random.default_rng(1)
    a, sa = rng.integers(0, 256, (5, 48), dtype=np.uint8), rng.integers(120, 134, (5, 3), dtype=np.uint8)
    w, sw = rng.integers(0, 256, (2, 4, 48), dtype=np.uint8), rng.integers(120, 134, (2, 4, 3), dtype=np.uint8)
    off, g = [0, 2, 5], np.array([8, 1, 6, 3, 5])
    out, mag = oracle.grouped_gemm_mx4(a, sa, w, sw, off, g, 2)
    for i, e in enumerate([0, 0, 1, 1, 1]):
        for n in range(4):
            v = 0.0
            for b in range(3):
                ca = oracle.e2m1_value(oracle.unpack_mx(a[g[i] // 2]))[32 * b:32 * b + 32]
                cw = oracle.e2m1_value(oracle.unpack_mx(w[e, n]))[32 * b:32 * b + 32]
                v += (ca * cw).sum() * 2.0 ** (int(sa[g[i] // 2, b]) + int(sw[e, n, b]) - 254)
            assert out[i, n] == v and mag[i, n] >= abs(v)


def case(T=7, E=6, k=3, H=5, seed=0, drop=True):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E))
    ids, _ = oracle.route_topk(logits.astype(np.float32), k, True)
    _, pos, _ = oracle.permute_pairs(ids, E)
    pos = np.array(pos)
    if drop:
        pos[[2, 9]] = [-1, 1000]
    return rng, logits, ids, pos, rng.standard_normal((T * k, H)), rng.standard_normal((T, H))


def test_dispatch_and_combine_by_loops():
    rng, logits, ids, pos, rows, x = case()
    w = rng.random((7, 3))
    got = dispatch.dispatch(x, pos, 3, rows, w)
    y = dispatch.combine(rows, pos, 3, w)
    want, wy = rows.copy(), np.zeros((7, 5))
    for p, at in enumerate(pos):
        if 0 <= at < 21:
            want[at] = w[p // 3, p % 3] * x[p // 3]
            wy[p // 3] += w[p // 3, p % 3] * rows[at]
    assert np.array_equal(got, want) and np.allclose(y, wy, rtol=0, atol=1e-14)


@pytest.mark.parametrize("renorm", [True, False])
def test_gradients_by_differences(renorm):
    rng, logits, ids, pos, rows, dy = case(seed=3)

    def loss(logits, rows):
        return (dispatch.combine(rows, pos, 3, dispatch.route_weights(logits, ids, renorm)) * dy).sum()

    w = dispatch.route_weights(logits, ids, renorm)
    drows, dw = dispatch.combine_backward(dy, rows, pos, 3, w)
    dl = dispatch.route_backward(logits, ids, dw, renorm)
    h = 1e-6
    for grad, arg in ((dl, 0), (drows, 1)):
        for i in np.ndindex(grad.shape):
            d = np.zeros_like(grad)
            d[i] = h
            args = [logits, rows]
            hi = list(args)
            lo = list(args)
            hi[arg], lo[arg] = args[arg] + d, args[arg] - d
            assert abs((loss(*hi) - loss(*lo)) / (2 * h) - grad[i]) < 1e-8
    # and a dispatch's gradient is the combine of the rows' gradient
    g = rng.standard_normal(rows.shape)
    dx = dispatch.combine(g, pos, 3, w)
    x = rng.standard_normal(dy.shape)
    d = np.zeros_like(x)
    d[4, 2] = 1.0
    base = np.zeros_like(rows)
    assert np.isclose((dispatch.dispatch(x + d, pos, 3, base, w) * g).sum()
                      - (dispatch.dispatch(x, pos, 3, base, w) * g).sum(), dx[4, 2])
