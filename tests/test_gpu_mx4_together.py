"""The MXFP4 operators and dispatch as they are used: a layer with 4-bit activations, a training
step through a trainable router; and their largest places."""

import numpy as np
import pytest
import torch

import oracle
from oracle import dispatch
from parity import half_spacing
from test_gpu_mx4_gemm import tolerance

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def raw(t):
    return t.cpu().numpy()


def randn(*shape, seed=0):
    return torch.randn(*shape, device=DEV, generator=torch.Generator(DEV).manual_seed(seed))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 96), (5, 16, 4, 288, 128), (60, 4, 2, 256, 160),
                                       (300, 2, 1, 512, 256)])
def test_layer_of_four_bits(gpu_lib, T, E, k, H, I):
    """Routing, both products on MXFP4, combine: each on what the others gave it."""
    x = randn(T, H, seed=1).bfloat16()
    gu = gpu_lib.quantize_mxfp4(randn(E, 2 * I, H, seed=2) * 0.1)
    dn = gpu_lib.quantize_mxfp4(randn(E, H, I, seed=3) * 0.1)
    logits = randn(T, E, seed=4)
    r = gpu_lib.route_permute(logits, k)
    P = T * k
    h = gpu_lib.grouped_gemm_mx4(x, None, *gu, r["offsets"], P, gather=r["sorted_pair"], gather_div=k,
                                 swiglu=True, out_dtype=torch.float16)
    rows = gpu_lib.grouped_gemm_mx4(h, None, *dn, r["offsets"], P, out_dtype=torch.float32)
    y = gpu_lib.moe_combine(rows, r["pair_pos"], k, w=r["w"], y_dtype=torch.float32)
    # the same products scattered to pair order, and combined in that order
    pairs = gpu_lib.grouped_gemm_mx4(h, None, *dn, r["offsets"], P, scatter=r["sorted_pair"],
                                     out_dtype=torch.float32)
    order = torch.arange(P, dtype=torch.int32, device=DEV)
    assert torch.equal(gpu_lib.moe_combine(pairs, order, k, w=r["w"], y_dtype=torch.float32), y)
    off, sp = raw(r["offsets"]), raw(r["sorted_pair"])
    ref, mag = oracle.grouped_gemm_mx4(*oracle.quantize_mxfp4(host(x)), raw(gu[0]), raw(gu[1]), off,
                                       sp, k, True)
    assert (np.abs(host(h) - ref) <= tolerance(ref, mag, H, "f16", True)).all()
    ref, mag = oracle.grouped_gemm_mx4(*oracle.quantize_mxfp4(host(h)), raw(dn[0]), raw(dn[1]), off)
    assert (np.abs(host(rows) - ref) <= tolerance(ref, mag, I, "f32", False)).all()
    pos, w = raw(r["pair_pos"]), host(r["w"])
    ref = dispatch.combine(host(rows), pos, k, w)
    mag = dispatch.combine(np.abs(host(rows)), pos, k, w)
    assert (np.abs(host(y) - ref) <= (k + 1) * U * mag + half_spacing(ref, "f32")).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_training_step_through_the_router(gpu_lib, renorm):
    """y = combine(experts(dispatch(x)), w(logits)) with one frozen NF4 projection an expert:
    the gradients for x and the logits, by the formula and by differences of the loss."""
    T, E, k, H = 37, 8, 3, 128
    x = randn(T, H, seed=1).half()
    packed, absmax = gpu_lib.quantize(randn(E, H, H, seed=2) * 0.1)
    logits, gy = randn(T, E, seed=3), randn(T, H, seed=4)
    r = gpu_lib.route_permute(logits, k, renormalize=renorm)
    rows = gpu_lib.moe_dispatch(x, r["pair_pos"], k)
    out = gpu_lib.grouped_gemm(rows, packed, absmax, r["offsets"], T * k, out_dtype=torch.float32)
    y = gpu_lib.moe_combine(out, r["pair_pos"], k, w=r["w"])
    d_out, dw = gpu_lib.moe_combine_backward(gy, out, r["pair_pos"], k, w=r["w"],
                                             drows_dtype=torch.float16)
    d_rows = gpu_lib.grouped_dgrad(d_out, packed, absmax, r["offsets"], T * k, out_dtype=torch.float32)
    dx = gpu_lib.moe_combine(d_rows, r["pair_pos"], k)
    dlogits = gpu_lib.moe_route_backward(logits, r["ids"], dw, renormalize=renorm)

    W = np.stack([oracle.dequantize_blockwise(raw(packed)[e:e + 1], raw(absmax)[e:e + 1])[0]
                  for e in range(E)]).astype(np.float64)
    ids, hx, hl, hg = raw(r["ids"]).astype(int), host(x), host(logits), host(gy)

    def forward(hx, hl):
        w = dispatch.route_weights(hl, ids, renorm)
        return np.einsum("tk,tkh->th", w, np.einsum("tkhc,tc->tkh", W[ids], hx)), w

    ref, w = forward(hx, hl)
    # weights and rows are held to fp16 (2^-11 a factor) in the products: H terms of either sign
    scale = np.abs(ref).max()
    assert np.abs(host(y) - ref).max() <= 4 * 2.0 ** -11 * scale
    per = np.einsum("tkhc,tc->tkh", W[ids], hx)
    want_dw = np.einsum("tkh,th->tk", per, hg)
    assert np.abs(host(dw) - want_dw).max() <= 4 * 2.0 ** -11 * np.abs(want_dw).max()
    want_dl = dispatch.route_backward(hl, ids, want_dw, renorm)
    assert np.abs(host(dlogits) - want_dl).max() <= 8 * 2.0 ** -11 * np.abs(want_dw).max()
    want_dx = np.einsum("tk,tkhc,th->tc", w, W[ids], hg)
    assert np.abs(host(dx) - want_dx).max() <= 4 * 2.0 ** -11 * np.abs(want_dx).max()
    loss = lambda hx, hl: (forward(hx, hl)[0] * hg).sum()  # noqa: E731
    rng = np.random.default_rng(0)
    for grad, arg, at in ((want_dl, 1, hl), (want_dx, 0, hx)):
        for _ in range(6):
            i = tuple(rng.integers(0, n) for n in at.shape)
            if arg == 1:
                i = (i[0], ids[i[0], 0])
            d = np.zeros_like(at)
            d[i] = 1e-5
            hi, lo = ((hx + d, hl), (hx - d, hl)) if arg == 0 else ((hx, hl + d), (hx, hl - d))
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - grad[i]) <= 1e-6 * (1 + abs(grad[i]))


def values(codes, scales):
    """fp64 values on the GPU."""
    grid = torch.tensor([float(v) for v in oracle.e2m1_value(np.arange(16))], dtype=torch.float64,
                        device=DEV)
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1, 32)
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), scales.double() - 127)
    return (grid[c.int()] * s[..., None]).reshape(*codes.shape[:-1], -1)


def operands(E, P, N, K, seed=0):
    g = torch.Generator(DEV).manual_seed(seed)
    b = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device=DEV, generator=g)  # noqa: E731
    return (b(0, 256, P, K // 2), b(121, 131, P, K // 32), b(0, 256, E, N, K // 2),
            b(121, 131, E, N, K // 32))


def sampled(y, a, sa, w, sw, expert, picks, K):
    for i in picks:
        v, m = values(a[i], sa[i]), values(w[expert(i)], sw[expert(i)])
        ref, mag = (m @ v).cpu().numpy(), (m.abs() @ v.abs()).cpu().numpy()
        tol = (K / 32 + 8) * 2.0 ** -23 * mag + half_spacing(ref, "f16" if y.dtype == torch.float16
                                                             else "f32")
        assert (np.abs(host(y[i]) - ref) <= tol).all(), i


@pytest.mark.parametrize("rows,N", [(1, 2304), (80, 2304)])
def test_more_tiles_of_a_workgroup_than_are_looked_up_at_once(gpu_lib, rows, N):
    """1024 experts: 18 and 36 tiles a workgroup where 32 are looked up at a time."""
    E, K = 1024, 64
    P = E * rows
    a, sa, w, sw = operands(E, P, N, K)
    off = (torch.arange(E + 1, device=DEV) * rows).int()
    sa = sa - 8  # sums that fp16 holds
    y = gpu_lib.grouped_gemm_mx4(a, sa, w, sw, off, P, out_dtype=torch.float32)
    sampled(y, a, sa, w, sw, lambda i: i // rows, [0, 1, P // 3, P // 2 + 7, P - 2, P - 1], K)
    # and every row against one product an expert in fp32, exact up to its roundings
    for e in range(0, E, 37):
        at = slice(e * rows, (e + 1) * rows)
        v = values(a[at], sa[at]) @ values(w[e], sw[e]).t().contiguous()
        m = values(a[at], sa[at]).abs() @ values(w[e], sw[e]).abs().t().contiguous()
        assert ((y[at].double() - v).abs() <= (K / 32 + 9) * 2.0 ** -23 * m + 1e-30).all()


def test_outputs_beyond_32_bits(gpu_lib):
    P, N, K = 262400, 8208, 32  # 2.15e9 results
    a, sa, w, sw = operands(1, P, N, K)
    sa = sa - 10
    off = torch.tensor([0, P], dtype=torch.int32, device=DEV)
    y = gpu_lib.grouped_gemm_mx4(a, sa, w, sw, off, P, out_dtype=torch.float16)
    sampled(y, a, sa, w, sw, lambda i: 0, [0, P // 2, 261700, P - 1], K)
    rs = torch.ones(P, device=DEV)  # the way with places of their own
    z = gpu_lib.grouped_gemm_mx4(a, sa, w, sw, off, P, row_scale=rs, out_dtype=torch.float16)
    assert torch.equal(y, z)


@pytest.mark.parametrize("counts", [[1, 0, 2, 0, 3], [40, 0, 5, 0, 30], [100, 90, 0, 0, 220]])
def test_stacks_beyond_32_bits(gpu_lib, counts):
    E, N, K = 5, 16384, 131072  # 1 GiB of codes an expert
    P = sum(counts)
    a, sa, w, sw = operands(E, P, N, K)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    y = gpu_lib.grouped_gemm_mx4(a, sa, w, sw, off, P, out_dtype=torch.float32)
    ex = np.repeat(np.arange(E), counts)
    for i in (0, P - 1):
        for n0 in (0, N - 64):
            v, m = values(a[i], sa[i]), values(w[ex[i], n0:n0 + 64], sw[ex[i], n0:n0 + 64])
            ref, mag = (m @ v).cpu().numpy(), (m.abs() @ v.abs()).cpu().numpy()
            assert (np.abs(host(y[i, n0:n0 + 64]) - ref) <= (K / 32 + 8) * 2.0 ** -23 * mag
                    + half_spacing(ref, "f32")).all()


def test_blocks_beyond_32_bits(gpu_lib):
    R, K = 132000, 32768  # 4.3e9 values
    x = torch.empty(R, K, dtype=torch.bfloat16, device=DEV)
    x.view(torch.int16).copy_(torch.randint(-20000, 20000, (1, K), dtype=torch.int16, device=DEV).expand(R, K))
    x[-1] = torch.randn(K, device=DEV)
    c, s = gpu_lib.quantize_mxfp4(x)
    for i in (0, R // 2, R - 1):
        want, scales = oracle.quantize_mxfp4(host(x[i]))
        assert np.array_equal(raw(c[i]), want) and np.array_equal(raw(s[i]), scales)
    back = gpu_lib.dequantize_mxfp4(c[-3:], s[-3:], torch.float32)
    # some of these bits are NaNs: their blocks read back as NaN
    assert np.array_equal(host(back), oracle.dequantize_mxfp4(raw(c[-3:]), raw(s[-3:])), equal_nan=True)
    whole = gpu_lib.dequantize_mxfp4(c, s, torch.bfloat16)
    assert torch.equal(whole[-3:].isnan(), back.isnan())
    assert torch.equal(whole[-3:].nan_to_num(), back.bfloat16().nan_to_num())
    del whole
    ct, st = gpu_lib.quantize_mxfp4(x, transpose=True)  # [K, R / 2]
    for j in (0, K - 1):
        want, scales = oracle.quantize_mxfp4(host(x[:, j]))
        assert np.array_equal(raw(ct[j]), want) and np.array_equal(raw(st[j]), scales)


def test_rows_beyond_32_bits(gpu_lib):
    T, k, H = 70000, 8, 4096  # 2.3e9 elements of rows
    x = randn(T, H).bfloat16()
    pos = torch.randperm(T * k, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).int()
    rows = gpu_lib.moe_dispatch(x, pos, k)
    at = pos.long()
    for p in (0, T * k // 2, T * k - 1, int(torch.argmax(at)), int(torch.argmin(at))):
        assert torch.equal(rows[at[p]], x[p // k])
    w = torch.rand(T, k, device=DEV)
    y = gpu_lib.moe_combine(rows, pos, k, w=w, y_dtype=torch.float32)
    want = x[-5:].double() * w[-5:].double().sum(1, keepdim=True)
    assert ((y[-5:].double() - want).abs() <= (k + 2) * U * want.abs() * 2).all()
    # in the place of the rows; every row is its token's, so dw is the token's square
    drows, dw = gpu_lib.moe_combine_backward(x, rows, pos, k, w=w, drows=rows)
    sq = (x.double() ** 2).sum(1, keepdim=True).expand(T, k)
    assert ((dw.double() - sq).abs() <= (H / 8 + 17) * U * sq).all()
    for p in (0, T * k - 1, int(torch.argmax(at))):
        want = (x[p // k].double() * w[p // k, p % k].double())
        assert ((drows[at[p]].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -20)).all()
