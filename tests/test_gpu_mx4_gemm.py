"""The grouped product of two MXFP4 operands on the GPU against 64 bits.

Tolerance per element: the sums inside a block of 32 are exact (multiples of 1/4 below
1152); the blocks are added in fp32, at most one addition a block and eight more where waves
join, each off by at most 2^-23 of the terms' magnitudes (a matrix-unit sum may drop bits
instead of rounding).  So |y - ref| <= (K/32 + 8) 2^-23 sum|terms| plus half a step of y's
type.  SwiGLU: silu's slope is at most 1.1, and its exponential, reciprocal and products are
off by (|z| + 8) 2^-23 of the value.
"""

import numpy as np
import pytest
import torch

import oracle
from parity import half_spacing

pytestmark = pytest.mark.gpu
DEV = "cuda"
TT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def host(t):
    return t.detach().double().cpu().numpy()


def dev(a):
    return None if a is None else torch.as_tensor(a).to(DEV)


def operand(rng, *shape, K):
    """Codes and scales: any codes, scales within 2^12."""
    return (rng.integers(0, 256, (*shape, K // 2), dtype=np.uint8),
            rng.integers(120, 132, (*shape, K // 32), dtype=np.uint8))


def counts_to_offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def tolerance(ref, mag, K, out, swiglu):
    steps = (K / 32 + 8) * 2.0 ** -23
    if not swiglu:
        return steps * mag + half_spacing(ref, out)
    pre, m = mag
    z, u = np.split(pre, 2, axis=1)
    tz, tu = np.split(steps * m, 2, axis=1)
    s = np.abs(z / (1 + np.exp(-z)))
    return (1.1 * tz * (np.abs(u) + tu) + s * tu + (np.abs(z) + 8) * 2.0 ** -23 * np.abs(ref)
            + half_spacing(ref, out))


def check(y, ref, mag, K, out="f32", swiglu=False):
    tol = tolerance(ref, mag, K, out, swiglu)
    bad = ~(np.abs(host(y) - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], (np.abs(host(y) - ref) / tol).max())


def case(counts, N, K, seed=0, rows=None, k=None, scale=1.0):
    """Operands and offsets; with k pairs a token gather over ``rows`` tokens.  SwiGLU
    wants moderate sums: ``scale`` shifts the scale bytes."""
    rng = np.random.default_rng((seed, N, K, len(counts)))
    off = counts_to_offsets(counts)
    P = int(off[-1])
    rows = P if rows is None else rows
    a, sa = operand(rng, rows, K=K)
    w, sw = operand(rng, len(counts), N, K=K)
    if scale != 1.0:
        sa = sa - np.uint8(-np.log2(scale))
    g = rng.integers(0, rows * k, P).astype(np.int32) if k else None
    return dict(a=a, sa=sa, w=w, sw=sw, off=off, P=P, g=g, k=k or 1, K=K)


def ref_of(c, swiglu=False):
    return oracle.grouped_gemm_mx4(c["a"], c["sa"], c["w"], c["sw"], c["off"], c["g"], c["k"], swiglu)


def run(lib, c, **kw):
    return lib.grouped_gemm_mx4(dev(c["a"]), dev(c["sa"]), dev(c["w"]), dev(c["sw"]), dev(c["off"]),
                                c["P"], gather=dev(c["g"]), gather_div=c["k"], **kw)


COUNTS = {"one": [1], "few": [1, 0, 2], "decode": [1] * 8 + [0] * 20 + [1],
          "edges": [15, 16, 17, 0, 31, 33], "tiles": [63, 64, 65, 0, 1], "large": [127, 129, 257],
          "long": [700], "many": [3] * 200}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K", [(64, 128), (272, 256), (160, 2880)])
def test_rows_of_experts(gpu_lib, name, N, K):
    if name in ("many", "large", "long") and K > 1000:
        N = 48
    c = case(COUNTS[name], N, K)
    ref, mag = ref_of(c)
    check(run(gpu_lib, c, out_dtype=torch.float32), ref, mag, K)


@pytest.mark.parametrize("E,picks", [(1000, [0, 63, 64, 65, 500, 999]), (1024, [1023]), (65, [64])])
def test_few_rows_of_many_experts(gpu_lib, E, picks):
    counts = np.zeros(E, dtype=int)
    counts[picks] = np.arange(1, len(picks) + 1)
    c = case(list(counts), 48, 96)
    assert c["P"] <= 32
    ref, mag = ref_of(c)
    check(run(gpu_lib, c, out_dtype=torch.float32), ref, mag, 96)


@pytest.mark.parametrize("counts", [[17, 0, 15], [16], [32], [1, 31], [0, 32, 0], [20, 12]])
def test_several_tiles_of_few_rows(gpu_lib, counts):
    for K in (96, 4096, 4128, 9216):
        c = case(counts, 48, K, rows=11, k=3)
        ref, mag = ref_of(c)
        check(run(gpu_lib, c, out_dtype=torch.float32), ref, mag, K)


@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 288, 480, 512, 544, 1056, 8192, 8224])
@pytest.mark.parametrize("counts", [[5], [70, 3], [300]])
def test_every_tail_of_k(gpu_lib, counts, K):
    c = case(counts, 32, K)
    ref, mag = ref_of(c)
    check(run(gpu_lib, c, out_dtype=torch.float32), ref, mag, K)


@pytest.mark.parametrize("N", [16, 32, 48, 240, 256, 272, 528])
@pytest.mark.parametrize("counts", [[2, 3], [40, 90], [280]])
def test_every_tail_of_n(gpu_lib, counts, N):
    c = case(counts, N, 160)
    ref, mag = ref_of(c)
    check(run(gpu_lib, c, out_dtype=torch.float32), ref, mag, 160)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts", [[1, 4], [150, 20], [260]])
def test_output_types(gpu_lib, counts, out):
    c = case(counts, 80, 256, scale=2.0 ** -6)
    ref, mag = ref_of(c)
    check(run(gpu_lib, c, out_dtype=TT[out]), ref, mag, 256, out)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts", [[1, 0, 4], [150, 20], [300]])
@pytest.mark.parametrize("N,K", [(32, 96), (96, 256), (544, 128)])
def test_swiglu(gpu_lib, counts, N, K, out):
    c = case(counts, N, K, scale=2.0 ** -8)
    ref, mag = ref_of(c, True)
    check(run(gpu_lib, c, swiglu=True, out_dtype=TT[out]), ref, mag, K, out, True)


@pytest.mark.parametrize("counts", [[3, 0, 5], [100, 60, 0, 9], [300, 300]])
@pytest.mark.parametrize("swiglu", [False, True])
def test_gather_scatter_and_row_scale(gpu_lib, counts, swiglu):
    c = case(counts, 64, 160, rows=37, k=4, scale=2.0 ** -8)
    rng = np.random.default_rng(5)
    P = c["P"]
    perm = rng.permutation(P + 3)[:P].astype(np.int32)
    rs = rng.standard_normal(P).astype(np.float32)
    ref, mag = ref_of(c, swiglu)
    out = torch.full((P + 3, ref.shape[1]), 7.0, device=DEV)
    run(gpu_lib, c, swiglu=swiglu, row_scale=dev(rs), scatter=dev(perm), out=out)
    tol = tolerance(ref, mag, 160, "f32", swiglu)
    want, t = ref * rs[:, None], tol * np.abs(rs)[:, None] + half_spacing(ref * rs[:, None], "f32")
    got = host(out)
    assert (np.abs(got[perm] - want) <= t).all()
    rest = np.setdiff1d(np.arange(P + 3), perm)
    assert (got[rest] == 7).all()


@pytest.mark.parametrize("P,rows", [(64, 64), (300, 300)])
def test_scatter_outside_writes_nothing(gpu_lib, P, rows):
    c = case([P], 32, 128)
    sc = np.arange(P, dtype=np.int32)
    sc[::3] = -1
    sc[1::3] += 100000
    out = torch.full((rows + 1, 32), 7.0, device=DEV)
    run(gpu_lib, c, scatter=dev(sc), out=out[:rows])
    ref, mag = ref_of(c)
    got = host(out)
    keep = np.arange(2, P, 3)
    assert (np.abs(got[keep] - ref[keep]) <= tolerance(ref, mag, 128, "f32", False)[keep]).all()
    assert (np.delete(got, keep, 0) == 7).all()


@pytest.mark.parametrize("counts", [[2, 3], [90, 30], [260, 10]])
def test_rows_behind_the_last_are_left(gpu_lib, counts):
    c = case(counts, 48, 128)
    P = c["P"]
    ref, mag = ref_of(c)
    a = np.concatenate([c["a"], c["a"]])
    sa = np.concatenate([c["sa"], c["sa"]])
    out = torch.full((2 * P, 48), 7.0, device=DEV)
    gpu_lib.grouped_gemm_mx4(dev(a), dev(sa), dev(c["w"]), dev(c["sw"]), dev(c["off"]), 2 * P, out=out)
    check(out[:P], ref, mag, 128)
    assert (out[P:] == 7).all()
    # and rows that the offsets have beyond P
    out.fill_(7.0)
    gpu_lib.grouped_gemm_mx4(dev(a), dev(sa), dev(c["w"]), dev(c["sw"]), dev(c["off"]), P - 1,
                             out=out[:P])
    assert np.abs(host(out[:P - 1]) - ref[:P - 1]).max() <= tolerance(ref, mag, 128, "f32", False).max()
    assert (out[P - 1:] == 7).all()


def test_gathered_indices_outside_stay_in_memory(gpu_lib):
    for P in (6, 300):
        c = case([P], 32, 96)
        g = np.arange(P, dtype=np.int32)
        g[1], g[2], g[3] = -1, 2 ** 31 - 1, P
        out = gpu_lib.grouped_gemm_mx4(dev(c["a"]), dev(c["sa"]), dev(c["w"]), dev(c["sw"]),
                                       dev(c["off"]), P, gather=dev(g), out_dtype=torch.float32)
        ref, mag = ref_of(c)
        ok = np.r_[0, 4:P]
        assert (np.abs(host(out)[ok] - ref[ok]) <= tolerance(ref, mag, 96, "f32", False)[ok]).all()


@pytest.mark.parametrize("counts", [[3, 4], [140, 40], [290]])
def test_scales_without_a_value(gpu_lib, counts):
    K, N = 224, 48
    c = case(counts, N, K)
    clean = ref_of(c)
    c["sa"][2, 3] = 255
    c["sw"][0, 7, 6] = 255
    y = host(run(gpu_lib, c, out_dtype=torch.float32))
    nan = np.zeros(y.shape, bool)
    nan[2] = True
    nan[:counts[0], 7] = True
    assert np.array_equal(np.isnan(y), nan)
    ref, mag = clean
    assert (np.abs(y - ref) <= tolerance(ref, mag, K, "f32", False))[~nan].all()


@pytest.mark.parametrize("counts", [[3], [200]])
def test_smallest_and_largest_scales(gpu_lib, counts):
    K, N = 160, 32
    c = case(counts, N, K)
    rng = np.random.default_rng(2)
    c["sa"] = rng.integers(0, 4, c["sa"].shape, dtype=np.uint8)
    c["sw"] = rng.integers(225, 254, c["sw"].shape, dtype=np.uint8)
    ref, mag = ref_of(c)
    check(run(gpu_lib, c, out_dtype=torch.float32), ref, mag, K)
    c["sw"] = np.zeros_like(c["sw"])  # products below every fp32 number
    assert (host(run(gpu_lib, c, out_dtype=torch.float32)) == 0).all()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts,rows,k", [([1, 0, 1], 1, 2), ([4, 9, 0, 3], 8, 2),
                                           ([100, 156], 64, 4), ([300], 300, 1)])
@pytest.mark.parametrize("K", [96, 256, 2048])
def test_rows_quantised_by_the_call(gpu_lib, t, counts, rows, k, K):
    """The same bits as with codes made before."""
    c = case(counts, 64, K, rows=rows, k=k)
    x = torch.randn(rows, K, device=DEV, generator=torch.Generator(DEV).manual_seed(K)).to(TT[t])
    x[0, 40:64] = 0
    if rows > 3:
        x[3, 5] = float("inf")
    codes, s = gpu_lib.quantize_mxfp4(x)
    args = (dev(c["w"]), dev(c["sw"]), dev(c["off"]), c["P"])
    kw = dict(gather=dev(c["g"]), gather_div=k, out_dtype=torch.float32)
    one = gpu_lib.grouped_gemm_mx4(x, None, *args, **kw)
    two = gpu_lib.grouped_gemm_mx4(codes, s, *args, **kw)
    assert torch.equal(torch.isnan(one), torch.isnan(two))
    assert torch.equal(torch.nan_to_num(one), torch.nan_to_num(two))
    c["a"], c["sa"] = codes.cpu().numpy(), s.cpu().numpy()
    ref, mag = ref_of(c)
    ok = ~np.isnan(ref)
    assert (np.abs(host(one) - ref) <= tolerance(ref, mag, K, "f32", False))[ok].all()
    assert np.isnan(host(one))[~ok].all()


def test_the_input_gradient_through_the_transposed_stack(gpu_lib):
    """dx = dy W with dy quantised along N and the stack along its rows: the formula's value,
    and the slope of the product <dy, a W'> in a, which is linear."""
    g = torch.Generator(DEV).manual_seed(3)
    E, N, K, counts = 3, 192, 160, [30, 0, 61]
    w = torch.randn(E, N, K, device=DEV, generator=g) * 0.1
    off = dev(counts_to_offsets(counts))
    P = 91
    dy = torch.randn(P, N, device=DEV, generator=g)
    wt, st = gpu_lib.quantize_mxfp4(w, transpose=True)
    dx = gpu_lib.grouped_gemm_mx4(dy, None, wt, st, off, P, out_dtype=torch.float32)
    d, s = gpu_lib.quantize_mxfp4(dy)
    ref, mag = oracle.grouped_gemm_mx4(d.cpu().numpy(), s.cpu().numpy(), wt.cpu().numpy(),
                                       st.cpu().numpy(), off.cpu().numpy())
    check(dx, ref, mag, N)
    dv = oracle.dequantize_mxfp4(d.cpu().numpy(), s.cpu().numpy())
    wv = np.swapaxes(oracle.dequantize_mxfp4(wt.cpu().numpy(), st.cpu().numpy()), 1, 2)  # [E, N, K]
    ex = np.repeat(np.arange(E), counts)
    rng = np.random.default_rng(0)
    a = rng.standard_normal((P, K))
    loss = lambda a: sum((dv[i] * (wv[ex[i]] @ a[i])).sum() for i in range(P))  # noqa: E731
    for _ in range(8):
        i, j = rng.integers(P), rng.integers(K)
        h = np.zeros_like(a)
        h[i, j] = 1.0
        slope = (loss(a + h) - loss(a - h)) / 2
        assert abs(slope - host(dx)[i, j]) <= tolerance(ref, mag, N, "f32", False)[i, j] + 1e-9


def test_stacks_at_odd_places(gpu_lib):
    """Scales at every byte offset, one expert of a larger stack, codes at 16 bytes."""
    for counts in ([4], [200]):
        c = case(counts, 32, 416)
        ref, mag = ref_of(c)
        for at in range(1, 4):
            flat = torch.zeros(at + c["sw"].size, dtype=torch.uint8, device=DEV)
            flat[at:] = dev(c["sw"]).view(-1)
            fa = torch.zeros(at + c["sa"].size, dtype=torch.uint8, device=DEV)
            fa[at:] = dev(c["sa"]).view(-1)
            wf = torch.zeros(16 + c["w"].size, dtype=torch.uint8, device=DEV)
            wf[16:] = dev(c["w"]).view(-1)
            y = gpu_lib.grouped_gemm_mx4(dev(c["a"]), fa[at:].view(c["sa"].shape),
                                         wf[16:].view(c["w"].shape), flat[at:].view(c["sw"].shape),
                                         dev(c["off"]), c["P"], out_dtype=torch.float32)
            check(y, ref, mag, 416)


@pytest.mark.parametrize("counts", [[2, 5], [130, 140], [600]])
def test_captured_and_replayed(gpu_lib, counts):
    c = case(counts, 96, 320, rows=50, k=3)
    x = torch.randn(50, 320, device=DEV).bfloat16()
    args = [dev(c["w"]), dev(c["sw"]), dev(c["off"]), c["P"]]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out = torch.empty(c["P"], 96, device=DEV)
    call = lambda: gpu_lib.grouped_gemm_mx4(x, None, *args, gather=g, gather_div=3, out=out,  # noqa: E731
                                            workspace=ws)
    g = dev(c["g"])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        x.copy_(torch.randn(50, 320, device=DEV))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = gpu_lib.grouped_gemm_mx4(x, None, *args, gather=g, gather_div=3,
                                        out_dtype=torch.float32)
        assert torch.equal(got, want), i


def test_two_streams_at_once(gpu_lib):
    cs = [case([90, 200], 160, 512, seed=1), case([3, 1, 0, 2], 160, 512, seed=2)]
    want = [run(gpu_lib, c, out_dtype=torch.float32) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(10):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(gpu_lib, c, out_dtype=torch.float32))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_refusals_of_the_binding(gpu_lib):
    c = case([4, 4], 32, 64)
    a, sa, w, sw, off = (dev(c[k]) for k in ("a", "sa", "w", "sw", "off"))
    f = gpu_lib.grouped_gemm_mx4
    for bad in (lambda: f(a[:, :16], sa, w, sw, off, 8), lambda: f(a, sa[:, :1], w, sw, off, 8),
                lambda: f(a, sa, w, sw[:1], off, 8), lambda: f(a, sa, w, sw, off[:2], 8),
                lambda: f(a, sa, w[0], sw, off, 8), lambda: f(a.cpu(), sa, w, sw, off, 8),
                lambda: f(a, sa, w, sw, off, 8, out=torch.empty(8, 31, device=DEV)),
                lambda: f(a, sa, w, sw, off, 8, gather=off),
                lambda: f(torch.randn(8, 96, device=DEV), None, w, sw, off, 8)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(a.float()[:, :32], sa, w, sw, off, 8), lambda: f(a, sa, w, sw, off.long(), 8),
                lambda: f(torch.randn(8, 64, device=DEV).double(), None, w, sw, off, 8)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(gpu_lib.Nf4MoeError):
        f(a, sa, w, sw, off, 9)  # a has 8 rows
    with pytest.raises(gpu_lib.Nf4MoeError):
        f(torch.randn(64, 64, device=DEV), None, w, sw, off, 64,
          workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert f(a[:0], sa[:0], w, sw, off, 0).shape == (0, 32)
