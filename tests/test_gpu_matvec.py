"""4-bit matrix-vector products on the GPU against 64 bits.

Tolerance per element, from the number of roundings: each product, scale and sum is
fp32 (a matrix-unit sum may drop bits instead of rounding: 2^-23 a step); a
sum over K goes through at most K/32 partial sums in one accumulator plus 64 for the
32 products of a step, the waves and the bias.  nf4 levels carry 2^-22.  So
|y - ref| <= (K/32 + 64) 2^-23 sum|W x| plus half a step of y's type.
"""

import numpy as np
import pytest
import torch

import oracle
from parity import half_spacing

pytestmark = pytest.mark.gpu
DEV = "cuda"
TT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(qt, group, T, N, K, xt="bf16", sd="f32", zeros=True, seed=0):
    rng = np.random.default_rng((seed, T, N, K))
    x = torch.from_numpy(rng.standard_normal((T, K), dtype=np.float32)).to(TT[xt])
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    z = None
    if qt == "mxfp4":
        s = rng.integers(112, 124, (N, K // group), dtype=np.uint8)
        st = torch.from_numpy(s)
    else:
        st = torch.from_numpy(rng.uniform(0.01, 0.1, (N, K // group)).astype(np.float32))
        st = st.to(TT[sd])
        s = st.float().numpy()
        if qt == "int4" and zeros:
            z = rng.integers(0, 16, (N, K // group), dtype=np.uint8)
    return x, codes, st, s, z


def run(lib, x, codes, st, z, qt, group, **kw):
    g = lambda a: None if a is None else torch.as_tensor(a).to(DEV)  # noqa: E731
    return lib.nbit_matvec(g(x), g(codes), g(st), quant_type=qt, group=group, zeros=g(z), **kw)


def check(y, ref, mag, K, out):
    y = y.float().cpu().numpy().astype(np.float64)
    tol = (K / 32 + 64) * 2.0 ** -23 * mag + half_spacing(ref, out)
    bad = np.abs(y - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], (np.abs(y - ref) / tol).max())


FORMATS = [("nf4", 64), ("fp4", 64), ("int4", 32), ("int4", 64), ("int4", 128), ("mxfp4", 32)]


@pytest.mark.parametrize("qt,group", FORMATS)
@pytest.mark.parametrize("T", [1, 4, 16, 37])
def test_formats(gpu_lib, qt, group, T):
    N, K = 100, 1152
    x, codes, st, s, z = make(qt, group, T, N, K)
    ref, mag = oracle.matvec(x.float().numpy(), codes, s, qt, group, z)
    check(run(gpu_lib, x, codes, st, z, qt, group, out_dtype=torch.float32), ref, mag, K, "f32")


@pytest.mark.parametrize("qt,group,K", [("nf4", 64, 64), ("nf4", 64, 192), ("fp4", 64, 4160),
                                        ("int4", 32, 32), ("int4", 32, 96), ("int4", 128, 128),
                                        ("int4", 64, 8256), ("mxfp4", 32, 32), ("mxfp4", 32, 2880),
                                        ("mxfp4", 32, 16416), ("nf4", 64, 20480)])
@pytest.mark.parametrize("N", [1, 15, 17, 130])
def test_ragged_sizes(gpu_lib, qt, group, K, N):
    for T in (1, 3, 8, 17):
        x, codes, st, s, z = make(qt, group, T, N, K, xt="f16")
        ref, mag = oracle.matvec(x.float().numpy(), codes, s, qt, group, z)
        check(run(gpu_lib, x, codes, st, z, qt, group, out_dtype=torch.float32), ref, mag, K, "f32")


@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sd", ["bf16", "f16", "f32"])
def test_types_bias_and_no_zeros(gpu_lib, xt, out, sd):
    T, N, K = 2, 77, 640
    x, codes, st, s, z = make("int4", 32, T, N, K, xt=xt, sd=sd, zeros=False)
    b = np.random.default_rng(3).standard_normal(N).astype(np.float32)
    ref, mag = oracle.matvec(x.float().numpy(), codes, s, "int4", 32, None, b)
    y = run(gpu_lib, x, codes, st, None, "int4", 32, bias=torch.from_numpy(b).to(DEV),
            out_dtype=TT[out])
    assert y.dtype == TT[out]
    check(y, ref, mag, K, out)


@pytest.mark.parametrize("N,K,T", [(40003, 256, 1), (40003, 256, 5), (70001, 128, 1), (70001, 128, 4),
                                   (9007, 256, 16), (9007, 4224, 1), (16401, 4224, 2),
                                   (16401, 4224, 9), (9007, 2112, 3), (5000, 4160, 33)])
@pytest.mark.parametrize("qt,group", [("nf4", 64), ("int4", 32), ("mxfp4", 32)])
def test_many_row_tiles(gpu_lib, qt, group, N, K, T):
    """More output rows than one pass of the grid takes, in rounds of one to four
    tiles; checked at the edges of the tiles and rounds and at some rows between."""
    x, codes, st, s, z = make(qt, group, T, N, K)
    y = run(gpu_lib, x, codes, st, z, qt, group, out_dtype=torch.float32)
    rng = np.random.default_rng(8)
    rows = np.unique(np.concatenate([np.arange(130), np.arange(4060, 4140), np.arange(N - 70, N),
                                     rng.integers(0, N, 300)]))
    ref, mag = oracle.matvec(x.float().numpy(), codes[rows], s[rows], qt, group,
                             None if z is None else z[rows])
    check(y[:, torch.from_numpy(rows).to(DEV)], ref, mag, K, "f32")


def test_quantised_stack_slice_and_untouched_neighbours(gpu_lib):
    """One expert of a quantised stack is a matrix; memory around y stays."""
    w = torch.randn(3, 50, 320, device=DEV, generator=torch.Generator(DEV).manual_seed(1)) * 0.02
    codes, absmax = gpu_lib.quantize(w)
    x = torch.randn(5, 320, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).half()
    buf = torch.full((7, 50), 3.0, device=DEV)
    gpu_lib.nbit_matvec(x, codes[1], absmax[1], out=buf[1:6])
    ref, mag = oracle.matvec(x.float().cpu().numpy(), codes[1].cpu().numpy(),
                             absmax[1].cpu().numpy(), "nf4", 64)
    check(buf[1:6], ref, mag, 320, "f32")
    assert torch.all(buf[0] == 3.0) and torch.all(buf[6] == 3.0)


@pytest.mark.parametrize("qt,group,K", [("int4", 128, 128), ("int4", 32, 96), ("mxfp4", 32, 32),
                                        ("mxfp4", 32, 160), ("nf4", 64, 64)])
def test_scales_zeros_bias_and_out_at_any_element(gpu_lib, qt, group, K):
    """Scales, zeros, bias and y begin one row into larger arrays: only their own
    element's alignment."""
    T, N = 3, 21
    sd = "f16" if qt == "int4" else "f32"
    x, codes, st, s, z = make(qt, group, T, N + 1, K, sd=sd)
    b = torch.randn(N + 1, generator=torch.Generator().manual_seed(4))
    out = torch.zeros((T + 1) * N + 1, dtype=torch.bfloat16, device=DEV)
    y = out[1:1 + T * N].view(T, N)
    gpu_lib.nbit_matvec(x.to(DEV), torch.as_tensor(codes[1:]).to(DEV), st.to(DEV)[1:], quant_type=qt,
                        group=group, zeros=None if z is None else torch.as_tensor(z).to(DEV)[1:],
                        bias=b.to(DEV)[1:], out=y)
    ref, mag = oracle.matvec(x.float().numpy(), codes[1:], s[1:], qt, group,
                             None if z is None else z[1:], b.numpy()[1:])
    check(y, ref, mag, K, "bf16")
    assert out[0] == 0 and torch.count_nonzero(out[1 + T * N:]) == 0


def test_zero_activations_and_zero_scales(gpu_lib):
    x, codes, st, s, z = make("nf4", 64, 3, 33, 128)
    x[1] = 0
    y = run(gpu_lib, x, codes, st, z, "nf4", 64, out_dtype=torch.float32)
    assert torch.count_nonzero(y[1]) == 0 and torch.count_nonzero(y[0]) > 0
    assert torch.count_nonzero(run(gpu_lib, x, codes, st * 0, z, "nf4", 64)) == 0


@pytest.mark.parametrize("qt,group", FORMATS)
def test_non_finite_inputs_stay_in_their_row_and_column(gpu_lib, qt, group):
    T, N, K = 5, 40, 256
    x, codes, st, s, z = make(qt, group, T, N, K)
    clean = run(gpu_lib, x, codes, st, z, qt, group, out_dtype=torch.float32)
    x[2, 7] = float("nan")
    x[3, 100] = float("inf")
    y = run(gpu_lib, x, codes, st, z, qt, group, out_dtype=torch.float32)
    assert torch.all(torch.isnan(y[2])) and not torch.any(torch.isfinite(y[3]))
    assert torch.equal(y[[0, 1, 4]], clean[[0, 1, 4]])
    x, codes, st, s, z = make(qt, group, T, N, K)
    st[9, 1] = 255 if qt == "mxfp4" else float("nan")
    y = run(gpu_lib, x, codes, st, z, qt, group, out_dtype=torch.float32)
    assert torch.all(torch.isnan(y[:, 9]))
    keep = [n for n in range(N) if n != 9]
    assert torch.equal(y[:, keep], clean[:, keep])


def test_small_activations_keep_their_bits(gpu_lib):
    """fp16 subnormals go through the matrix unit as they are."""
    x, codes, st, s, z = make("fp4", 64, 2, 40, 128, xt="f16")
    x = (x.float() * 2.0 ** -20).half()
    ref, mag = oracle.matvec(x.float().numpy(), codes, s, "fp4", 64)
    check(run(gpu_lib, x, codes, st, z, "fp4", 64, out_dtype=torch.float32), ref, mag, 128, "f32")


def test_same_result_every_call(gpu_lib):
    x, codes, st, s, z = make("nf4", 64, 16, 333, 2048)
    y = run(gpu_lib, x, codes, st, z, "nf4", 64, out_dtype=torch.float32)
    for _ in range(2):
        assert torch.equal(run(gpu_lib, x, codes, st, z, "nf4", 64, out_dtype=torch.float32), y)


def test_stream_and_graph_replay(gpu_lib):
    x, codes, st, s, z = make("int4", 128, 3, 257, 1024)
    d = [torch.as_tensor(v).to(DEV) for v in (x, codes, st, z)]
    call = lambda out=None: gpu_lib.nbit_matvec(d[0], d[1], d[2], quant_type="int4", group=128,  # noqa: E731
                                                zeros=d[3], out=out)
    out = torch.empty((3, 257), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, call())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for i in range(3):
        d[0].copy_(torch.randn(3, 1024, device=DEV, generator=torch.Generator(DEV).manual_seed(i)))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call())


def test_binding_refuses_on_the_gpu(gpu_lib):
    x, codes, st, s, z = make("nf4", 64, 2, 8, 128)
    x, codes, st = x.to(DEV), torch.as_tensor(codes).to(DEV), st.to(DEV)
    for bad in (dict(scales=st[:, :1].contiguous()), dict(codes=codes[:, :32].contiguous()),
                dict(scales=st.cpu()), dict(out=torch.empty(2, 9, device=DEV)),
                dict(x=x.t().contiguous().t()), dict(bias=torch.zeros(9, device=DEV)),
                dict(zeros=torch.zeros(8, 3, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            gpu_lib.nbit_matvec(**dict(dict(x=x, codes=codes, scales=st), **bad))
    with pytest.raises(TypeError):
        gpu_lib.nbit_matvec(x, codes.to(torch.int32), st)
    with pytest.raises(gpu_lib.Nf4MoeError):
        gpu_lib.nbit_matvec(x.float(), codes, st)
