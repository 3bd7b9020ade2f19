"""The MXFP4 product where its places end: codes and scales far behind 2^31 bytes, and offsets
beyond the call's rows.  Tolerances as in test_gpu_mx4_gemm, each element with its own."""

import numpy as np
import pytest
import torch

from parity import half_spacing
from test_gpu_mx4_gemm import DEV, case, check, dev, host, ref_of
from test_gpu_mx4_together import operands, values
from test_gpu_mx4_wide import wide

pytestmark = pytest.mark.gpu


def check_columns(y, i, n0, n1, a, sa, w, sw, K):
    v, m = values(a, sa), values(w[n0:n1], sw[n0:n1])
    ref, mag = (m @ v).cpu().numpy(), (m.abs() @ v.abs()).cpu().numpy()
    tol = (K / 32 + 8) * 2.0 ** -23 * mag + half_spacing(ref, "f32")
    assert (np.abs(host(y[i, n0:n1]) - ref) <= tol).all(), (i, n0)


# rows that take 16-row tiles, 64-row ones and 256-row ones; scale rows of whole words and others
@pytest.mark.parametrize("P,N,K", [(3, 48000, 147456), (5, 200000, 32768), (40, 200000, 32768),
                                   (40, 200000, 32736), (150, 200000, 32768), (150, 200000, 32736)])
def test_one_matrix_of_more_than_2_gib(gpu_lib, P, N, K):
    assert 3 << 30 < N * K // 2 < 7 << 29
    a, sa, w, sw = operands(1, P, N, K)
    off = torch.tensor([0, P], dtype=torch.int32, device=DEV)
    y = gpu_lib.grouped_gemm_mx4(a, sa, w, sw, off, P, out_dtype=torch.float32)
    half = (1 << 31) // (K // 2)  # the row across 2^31 bytes
    for i in (0, P - 1):
        for n0 in (0, half - 32, N - 64):
            check_columns(y, i, n0, n0 + 64, a[i], sa[i], w[0], sw[0], K)


@pytest.mark.parametrize("P,N", [(20, 272), (300, 272), (12000, 272)])
@pytest.mark.parametrize("K", [32768, 32736])
def test_gathered_rows_behind_2_gib(gpu_lib, P, N, K):
    rows = 200000
    a, sa, w, sw = operands(1, rows, N, K)
    a, sa = a.view(rows, K // 2), sa.view(rows, K // 32)
    off = torch.tensor([0, P], dtype=torch.int32, device=DEV)
    half = (1 << 31) // (K // 2)
    g = torch.randint(0, rows, (P,), dtype=torch.int32, device=DEV,
                      generator=torch.Generator(DEV).manual_seed(P))
    at = {0: rows - 1, 1: half, 2: half - 1, 3: half + 1, P - 2: rows - 2, P - 1: 0}
    for i, r in at.items():
        g[i] = r
    y = gpu_lib.grouped_gemm_mx4(a, sa, w, sw, off, P, gather=g, out_dtype=torch.float32)
    for i in [*at, 7, P // 2, P - 3]:
        r = int(g[i])
        check_columns(y, i, 0, N, a[r], sa[r], w[0], sw[0], K)


@pytest.mark.parametrize("counts,less", [([2, 3, 4], 5), ([2, 3, 4], 1), ([9, 0, 12], 12), ([90, 30, 60], 75),
                                         ([90, 30, 60], 1), ([64, 64, 64], 64), ([260, 10, 7], 9)])
def test_offsets_beyond_the_rows(gpu_lib, counts, less):
    """Experts that end, or begin, behind P."""
    c = case(counts, 48, 128)
    P = c["P"] - less
    ref, mag = ref_of(c)
    out = torch.full((c["P"], 48), 7.0, device=DEV)
    gpu_lib.grouped_gemm_mx4(dev(c["a"]), dev(c["sa"]), dev(c["w"]), dev(c["sw"]), dev(c["off"]), P, out=out)
    check(out[:P], ref[:P], mag[:P], 128)
    assert (out[P:] == 7).all()


@pytest.mark.parametrize("N,K", [(48, 128), (272, 416)])
@pytest.mark.parametrize("behind,less", [([], 1), ([], 200), ([50, 70], 30), ([50, 70], 100), ([300, 0, 600], 700)])
def test_offsets_beyond_the_rows_of_large_tiles(gpu_lib, N, K, behind, less):
    c, _ = wide([40, 90, 280], N, K)
    rng = np.random.default_rng(9)
    last = int(c["off"][-1])
    more = sum(behind)
    # experts behind the ones that make the call large, of the first ones' weights
    off = np.r_[c["off"], last + np.cumsum(behind)].astype(np.int32)
    w = np.concatenate([c["w"], c["w"][:len(behind)]])
    sw = np.concatenate([c["sw"], c["sw"][:len(behind)]])
    a = np.concatenate([c["a"], rng.integers(0, 256, (more, K // 2), dtype=np.uint8)])
    sa = np.concatenate([c["sa"], rng.integers(120, 132, (more, K // 32), dtype=np.uint8)])
    P = last + more - less
    out = torch.full((last + more, N), 7.0, device=DEV)
    gpu_lib.grouped_gemm_mx4(dev(a), dev(sa), dev(w), dev(sw), dev(off), P, out=out)
    assert (out[P:] == 7).all()
    for lo in (0, max(0, P - 350)):  # the first rows, and the last
        hi = min(P, lo + 450)
        d = dict(c, a=a[lo:hi], sa=sa[lo:hi], w=w, sw=sw, off=np.clip(off, lo, hi) - lo)
        ref, mag = ref_of(d)
        check(out[lo:hi], ref, mag, K)
