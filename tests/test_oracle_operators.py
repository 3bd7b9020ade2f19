"""Pins of the oracle's operators around the routed experts: scalar loops, the
stacks' own dequantisers, differences and the singular-value polynomial."""

import numpy as np
import pytest

import oracle
from oracle import blocknorm, muon


def _rng(*key):
    return np.random.default_rng(key)


@pytest.mark.parametrize("qt", ["nf4", "fp4"])
def test_matvec_weight_is_the_stack_dequantised(qt):
    w = _rng(1).standard_normal((1, 6, 128)).astype(np.float32)
    codes, absmax = oracle.quantize_blockwise(w, quant_type=qt)
    got = oracle.matvec_weight(codes[0], absmax[0], qt, 64)
    want = oracle.dequantize_blockwise(codes, absmax, quant_type=qt)[0]
    assert np.allclose(got, want, rtol=2.0 ** -23, atol=0)


def test_matvec_weight_mxfp4_is_the_stack_dequantised():
    rng = _rng(2)
    blocks = rng.integers(0, 256, (5, 32), dtype=np.uint8)
    scales = rng.integers(118, 130, (5, 2), dtype=np.uint8)
    want = oracle.dequantize_mxfp4(blocks, scales)
    assert np.array_equal(oracle.matvec_weight(blocks, scales, "mxfp4", 32), want)


@pytest.mark.parametrize("zeros", [True, False])
def test_matvec_int4_scalar_loop(zeros):
    rng = _rng(3)
    N, K, G = 3, 64, 32
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = rng.standard_normal((N, K // G))
    z = rng.integers(0, 16, (N, K // G), dtype=np.uint8) if zeros else None
    x, b = rng.standard_normal((2, K)), rng.standard_normal(N)
    y, mag = oracle.matvec(x, codes, s, "int4", G, z, b)
    for t in range(2):
        for n in range(N):
            want, size = b[n], abs(b[n])
            for k in range(K):
                byte = int(codes[n, k // 2])
                c = byte >> 4 if k % 2 == 0 else byte & 15
                p = x[t, k] * s[n, k // G] * (c - (int(z[n, k // G]) if zeros else 8))
                want, size = want + p, size + abs(p)
            assert abs(y[t, n] - want) < 1e-12 * size and abs(mag[t, n] - size) < 1e-12 * size


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_block_norm_gradients_by_differences(post, pre, gate):
    rng = _rng(4, post, pre)
    T, H, eps, alpha, beta = 3, 8, 1e-3, 0.7, -0.6
    v = dict(residual=rng.standard_normal((T, H)), y=rng.standard_normal((T, H)))
    v["gate"] = {"none": np.ones(()), "token": rng.standard_normal((T, 1)),
                 "channel": rng.standard_normal((1, H))}[gate]
    v["w_post"] = rng.standard_normal(H) if post else None
    v["w_pre"] = rng.standard_normal(H) if pre else None
    dr, dh = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def loss(p):
        r, _ = blocknorm.post(p["residual"], p["y"], p["w_post"], p["gate"], alpha, beta, eps)
        out = (dr * r).sum()
        return out + (dh * blocknorm.pre(r, p["w_pre"], eps)).sum() if pre else out

    r, _ = blocknorm.post(v["residual"], v["y"], v["w_post"], v["gate"], alpha, beta, eps)
    got = blocknorm.backward(dh if pre else None, dr, r, v["y"], v["w_pre"], v["w_post"],
                             v["gate"], alpha, beta, eps)
    names = dict(residual="dresidual", y="dy", gate="dgate", w_pre="dw_pre", w_post="dw_post")
    for k, name in names.items():
        if v[k] is None or v[k].ndim == 0:
            assert name not in got
            continue
        num = np.zeros(v[k].size)
        for i in range(v[k].size):
            d = np.zeros(v[k].size)
            d[i] = 1e-5
            d = d.reshape(v[k].shape)
            num[i] = (loss(dict(v, **{k: v[k] + d})) - loss(dict(v, **{k: v[k] - d}))) / 2e-5
        value, size = got[name]
        # central differences: a third derivative times 1e-10 and 1e-16 / 1e-5
        assert np.allclose(np.ravel(value), num, atol=1e-7), name
        assert np.all(np.abs(value) <= size * (1 + 1e-12) + 1e-300), name


@pytest.mark.parametrize("shape", [(2, 1, 9), (3, 4, 33), (1, 16, 16), (2, 16, 5)])
def test_newton_schulz_is_its_polynomial_of_the_singular_values(shape):
    u = _rng(5).standard_normal(shape)
    c = (3.4445, -4.7750, 2.0315)
    U, S, V = np.linalg.svd(u, full_matrices=False)
    S = S / (np.sqrt((S ** 2).sum(1, keepdims=True)) + 1e-7)
    for _ in range(5):
        S = c[0] * S + c[1] * S ** 3 + c[2] * S ** 5
    want = (U * S[:, None, :]) @ V
    assert np.allclose(muon.newton_schulz(u, 5, c, 1e-7), want, atol=1e-10)
    t = muon.newton_schulz(u.transpose(0, 2, 1), 5, c, 1e-7).transpose(0, 2, 1)
    assert np.allclose(t, want, atol=1e-10)


def test_newton_schulz_of_zeros_is_zero():
    z = np.zeros((1, 2, 4))
    assert not muon.newton_schulz(z, 5, (3.4445, -4.775, 2.0315), 1e-7).any()
    assert not muon.newton_schulz(z, 5, (3.4445, -4.775, 2.0315), 0.0).any()
