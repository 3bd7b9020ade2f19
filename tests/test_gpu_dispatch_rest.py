"""Rows that no pair names: 0 in what the binding makes, as they were in what the caller gives.

The rows of the pairs are compared with the call on a buffer of the caller's, bit by bit; that
one is pinned against 64 bits in test_gpu_dispatch.
"""

import numpy as np
import pytest
import torch

from test_gpu_dispatch import DEV, TT, make

pytestmark = pytest.mark.gpu


def leave_nans(*shape, dtype):
    """Memory of this size, full of NaN, is what the next allocation gets."""
    t = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
    torch.cuda.synchronize()
    del t


def free_rows(c):
    pos = c["pos"].cpu().numpy()
    return np.setdiff1d(np.arange(c["R"]), pos)


def check_backward(lib, c, t):
    kept = torch.full((c["R"], c["H"]), 7.0, dtype=t, device=DEV)
    w = c["w"]
    lib.moe_combine_backward(c["x"], c["rows"], c["pos"], c["k"], w=w, drows=kept)
    leave_nans(c["R"], c["H"], dtype=t)
    drows, dw = lib.moe_combine_backward(c["x"], c["rows"], c["pos"], c["k"], w=w, drows_dtype=t)
    free = torch.from_numpy(free_rows(c)).to(DEV)
    assert (kept[free] == 7).all()
    kept[free] = 0
    assert torch.equal(drows, kept)
    assert torch.equal(dw, lib.moe_combine_backward(c["x"], c["rows"], c["pos"], c["k"], w=w,
                                                    need_drows=False)[1])


# rows padded, dropped, none free, one pair in many rows, several runs of rows, both ways of k
SHAPES = [(40, 4, 264, 200, 0.0), (40, 4, 264, 160, 0.3), (40, 4, 264, 160, 0.0), (1, 1, 2048, 333, 0.0),
          (3, 2, 1032, 4097, 0.2), (600, 8, 136, 6000, 0.1), (700, 6, 1448, 4201, 0.1),
          (2100, 2, 128, 42310, 0.5), (9, 3, 512, 31, 1.0), (2048, 4, 512, 8192, 0.0), (2300, 2, 1024, 5000, 0.3),
          # so short, or so many for their pairs, that all are cleared first
          (300, 4, 8, 1300, 0.1), (513, 8, 56, 4200, 0.4), (2100, 3, 128, 7000, 0.1)]


@pytest.mark.parametrize("T,k,H,R,drop", SHAPES)
@pytest.mark.parametrize("t", list(TT))
def test_gradient_of_rows_without_a_pair(gpu_lib, T, k, H, R, drop, t):
    check_backward(gpu_lib, make(T, k, H, R=R, drop=drop, xt="bf16", rt="f16"), TT[t])


def check_dispatch(lib, c, t, weighted=True):
    w = c["w"] if weighted else None
    kept = torch.full((c["R"], c["H"]), 7.0, dtype=t, device=DEV)
    lib.moe_dispatch(c["x"], c["pos"], c["k"], w=w, out=kept)
    leave_nans(c["R"], c["H"], dtype=t)
    rows = lib.moe_dispatch(c["x"], c["pos"], c["k"], w=w, rows=c["R"], out_dtype=t)
    free = torch.from_numpy(free_rows(c)).to(DEV)
    assert (kept[free] == 7).all()
    kept[free] = 0
    assert torch.equal(rows, kept)


@pytest.mark.parametrize("T,k,H,R,drop", SHAPES)
@pytest.mark.parametrize("t", list(TT))
def test_dispatched_rows_without_a_pair(gpu_lib, T, k, H, R, drop, t):
    c = make(T, k, H, R=R, drop=drop, xt="bf16")
    check_dispatch(gpu_lib, c, TT[t])
    check_dispatch(gpu_lib, c, TT[t], weighted=False)


@pytest.mark.parametrize("H", [8, 128])
def test_more_rows_than_workgroups_have_bits_for(gpu_lib, H):
    """Rows beyond 128 x 65536, and just as many."""
    for R in (128 * 65536, 128 * 65536 + 1):
        c = make(5, 2, H, R=40, rt="f16")
        far = torch.tensor([0, 1, 65535, 65536, R // 2, R // 2 + 33, R - 65537, R - 32, R - 2, R - 1],
                           dtype=torch.int32, device=DEV)
        rows = torch.zeros(R, H, dtype=torch.float16, device=DEV)
        rows[far.long()] = c["rows"][:10]
        leave_nans(R, H, dtype=torch.float16)
        drows, dw = gpu_lib.moe_combine_backward(c["x"], rows, far, 2, w=c["w"])
        del rows
        want = (c["w"].view(-1, 1) * c["x"].repeat_interleave(2, 0)).half()
        assert torch.equal(drows[far.long()], want)
        drows[far.long()] = 0
        assert not drows.view(torch.int32).any()
        del drows


def test_positions_at_any_word(gpu_lib):
    """Positions are read sixteen bytes at a time from wherever they begin."""
    c = make(1500, 3, 128, R=5000, drop=0.1)
    for at in (1, 2, 3):
        flat = torch.full((at + 4500,), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
        flat[at:] = c["pos"]
        check_backward(gpu_lib, dict(c, pos=flat[at:]), torch.float32)
        check_dispatch(gpu_lib, dict(c, pos=flat[at:]), torch.float32)


def test_a_sum_over_padded_rows(gpu_lib):
    """What a weight gradient makes of the rows: those of an expert with a padded end."""
    c = make(60, 2, 64, R=160)
    leave_nans(160, 64, dtype=torch.float32)
    drows, _ = gpu_lib.moe_combine_backward(c["x"], c["rows"], c["pos"], 2, w=c["w"])
    want = torch.zeros(160, 64, device=DEV)
    want[c["pos"].long()] = c["w"].view(-1, 1) * c["x"].repeat_interleave(2, 0)
    # one fp32 product a value, of which both sides have the same rounding
    assert torch.equal(drows.sum(0), want.sum(0))
    leave_nans(160, 64, dtype=torch.float32)
    rows = gpu_lib.moe_dispatch(c["x"], c["pos"], 2, rows=160)
    # the weight gradient's terms of the rows without a pair: 0 by 0
    terms = drows[:, :, None] * rows[:, None, :]
    assert torch.isfinite(terms).all()
    free = torch.from_numpy(free_rows(c)).to(DEV)
    assert len(free) == 40 and not terms[free].any()


def test_gradient_in_a_graph(gpu_lib):
    """Made while a graph is captured; positions change from replay to replay."""
    cs = [make(700, 3, 264, R=2400, drop=0.2, seed=i, rt="f16") for i in range(4)]
    c = {n: v.clone() if torch.is_tensor(v) else v for n, v in cs[0].items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        drows, dw = gpu_lib.moe_combine_backward(c["x"], c["rows"], c["pos"], 3, w=c["w"])
        sent = gpu_lib.moe_dispatch(c["x"], c["pos"], 3, rows=2400)
    for d in cs:
        for n in ("x", "rows", "pos", "w"):
            c[n].copy_(d[n])
        graph.replay()
        torch.cuda.synchronize()
        kept = torch.zeros(2400, 264, dtype=torch.float16, device=DEV)
        _, want = gpu_lib.moe_combine_backward(d["x"], d["rows"], d["pos"], 3, w=d["w"], drows=kept)
        assert torch.equal(drows, kept) and torch.equal(dw, want)
        rows = gpu_lib.moe_dispatch(d["x"], d["pos"], 3, out=torch.zeros(2400, 264, device=DEV))
        assert torch.equal(sent, rows)
