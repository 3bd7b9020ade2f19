"""The product's 256-row tiles on the GPU against 64 bits.

They run where there are rows and columns enough for the card, so an expert with many rows
stands behind the ones that are looked at, of which the last 70 rows are checked too.  Tolerances
as in test_gpu_mx4_gemm.
"""

import numpy as np
import pytest
import torch

from parity import half_spacing
from test_gpu_mx4_gemm import DEV, TT, case, dev, host, ref_of, run, tolerance

pytestmark = pytest.mark.gpu
SEEN = 70


def wide(counts, N, K, **kw):
    """A case with so many rows behind ``counts`` that 64-row tiles are more than two a
    compute unit, and the rows to look at."""
    places = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    tail = 64 * (places // ((N + 127) // 128) + 1)
    c = case([*counts, tail], N, K, **kw)
    assert c["P"] // min(len(counts) + 1, c["P"]) >= 80
    return c, np.r_[0:sum(counts), c["P"] - SEEN:c["P"]]


def seen(c, rows, swiglu=False):
    """The reference of those rows."""
    d = dict(c)
    d["off"] = np.r_[c["off"][:-1], c["off"][-2] + SEEN].astype(np.int32)
    if c["g"] is None:
        d["a"], d["sa"] = c["a"][rows], c["sa"][rows]
    else:
        d["g"] = c["g"][rows]
    return ref_of(d, swiglu)


def check(y, rows, ref, mag, K, out="f32", swiglu=False):
    tol = tolerance(ref, mag, K, out, swiglu)
    got = host(y)[rows]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], (np.abs(got - ref) / tol).max())


@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 256, 288, 480, 512, 544, 768, 1056, 2080])
@pytest.mark.parametrize("counts", [[5], [300, 0, 257]])
def test_every_tail_of_k(gpu_lib, counts, K):
    c, rows = wide(counts, 272, K)
    check(run(gpu_lib, c, out_dtype=torch.float32), rows, *seen(c, rows), K)


@pytest.mark.parametrize("N", [16, 32, 48, 240, 256, 272, 528])
@pytest.mark.parametrize("K", [96, 1024])
def test_every_tail_of_n(gpu_lib, N, K):
    c, rows = wide([40, 90, 280], N, K)
    check(run(gpu_lib, c, out_dtype=torch.float32), rows, *seen(c, rows), K)


@pytest.mark.parametrize("counts", [[1, 31, 32, 33, 63, 64, 65], [95, 97, 128, 129, 0, 160, 161],
                                    [191, 193, 224, 225], [255, 256, 257, 0, 511, 512, 513]])
@pytest.mark.parametrize("K", [128, 416])
def test_rows_of_experts(gpu_lib, counts, K):
    c, rows = wide(counts, 144, K)
    check(run(gpu_lib, c, out_dtype=torch.float32), rows, *seen(c, rows), K)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N,K", [(32, 96), (96, 256), (544, 128)])
def test_output_types(gpu_lib, N, K, swiglu, out):
    c, rows = wide([150, 20, 300], N, K, scale=2.0 ** -8)
    y = run(gpu_lib, c, swiglu=swiglu, out_dtype=TT[out])
    check(y, rows, *seen(c, rows, swiglu), K, out, swiglu)


@pytest.mark.parametrize("counts", [[3, 0, 5], [100, 60, 0, 9], [300, 300]])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [160, 256])
def test_gather_scatter_and_row_scale(gpu_lib, counts, swiglu, K):
    c, rows = wide(counts, 64, K, rows=37, k=4, scale=2.0 ** -8)
    rng = np.random.default_rng(5)
    P = c["P"]
    perm = rng.permutation(P + 3)[:P].astype(np.int32)
    left = rows[::7]
    perm[left[::2]] = -1 - perm[left[::2]]
    perm[left[1::2]] += P + 3
    rs = rng.standard_normal(P).astype(np.float32)
    ref, mag = seen(c, rows, swiglu)
    out = torch.full((P + 3, ref.shape[1]), 7.0, device=DEV)
    run(gpu_lib, c, swiglu=swiglu, row_scale=dev(rs), scatter=dev(perm), out=out)
    r = rs[rows][:, None]
    tol = tolerance(ref, mag, K, "f32", swiglu) * np.abs(r) + half_spacing(ref * r, "f32")
    there = (perm[rows] >= 0) & (perm[rows] < P + 3)
    got = host(out)
    assert (np.abs(got[perm[rows][there]] - (ref * r)[there]) <= tol[there]).all()
    rest = np.setdiff1d(np.arange(P + 3), perm)
    assert len(rest) == 3 + len(left) and (got[rest] == 7).all()


def test_indices_and_rows_outside(gpu_lib):
    """Gathered indices outside a, and rows behind the last expert's."""
    c, rows = wide([3, 300], 48, 96, rows=90, k=2)
    ref, mag = seen(c, rows)
    c["g"][:3] = -1, 2 ** 31 - 1, 180
    P = c["P"]
    g = np.r_[c["g"], np.zeros(500, np.int32)]
    out = torch.full((P + 500, 48), 7.0, device=DEV)
    gpu_lib.grouped_gemm_mx4(dev(c["a"]), dev(c["sa"]), dev(c["w"]), dev(c["sw"]), dev(c["off"]),
                             P + 500, gather=dev(g), gather_div=2, out=out)
    check(out, rows[3:], ref[3:], mag[3:], 96)
    assert (out[P:] == 7).all()


@pytest.mark.parametrize("K", [224, 1024])
def test_scales_without_a_value(gpu_lib, K):
    counts, N = [140, 40], 48
    c, rows = wide(counts, N, K)
    ref, mag = seen(c, rows)
    c["sa"][2, 3] = 255
    c["sw"][0, 7, 6] = 255
    y = host(run(gpu_lib, c, out_dtype=torch.float32))
    nan = np.zeros(y.shape, bool)
    nan[2] = True
    nan[:counts[0], 7] = True
    assert np.array_equal(np.isnan(y), nan)
    assert (np.abs(y[rows] - ref) <= tolerance(ref, mag, K, "f32", False))[~nan[rows]].all()


@pytest.mark.parametrize("K", [320, 512])
def test_captured_and_replayed(gpu_lib, K):
    """Rows quantised by the call, in a graph."""
    c, _ = wide([130, 140], 96, K, rows=50, k=3)
    x = torch.randn(50, K, device=DEV).bfloat16()
    args = [dev(c["w"]), dev(c["sw"]), dev(c["off"]), c["P"]]
    g = dev(c["g"])
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out = torch.empty(c["P"], 96, device=DEV)
    call = lambda: gpu_lib.grouped_gemm_mx4(x, None, *args, gather=g, gather_div=3, out=out,  # noqa: E731
                                            workspace=ws)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        x.copy_(torch.randn(50, K, device=DEV))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        codes, scales = gpu_lib.quantize_mxfp4(x)
        want = gpu_lib.grouped_gemm_mx4(codes, scales, *args, gather=g, gather_div=3,
                                        out_dtype=torch.float32)
        assert torch.equal(out, want), i


def test_two_streams_at_once(gpu_lib):
    cs = [wide([90, 200], 160, 512, seed=1)[0], wide([3, 1, 0, 2], 160, 416, seed=2)[0]]
    want = [run(gpu_lib, c, out_dtype=torch.float32) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append([run(gpu_lib, c, out_dtype=torch.float32) for _ in range(3)])
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert all(torch.equal(w, y) for y in many)
