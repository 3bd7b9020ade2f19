"""Refusals of the MXFP4 quantiser and product and of dispatch and combine: every bad
argument is found on the host, before anything is enqueued (CPU only, no kernel runs)."""

import pytest

from grouped_nf4_gemm_quantize_amd import binding


def at(i):
    return 0x100000 * (i + 1)  # distinct aligned pointers, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def refuse(lib, status, fn, defaults, changes):
    args = dict(defaults, **changes)
    assert list(args) == list(defaults)
    assert fn(*args.values()) == status, (changes, lib.nf4moe_last_error())
    assert lib.nf4moe_last_error()


QUANT = dict(x=at(0), xd=1, E=2, R=64, K=96, tr=0, codes=at(1), scales=at(2), stream=None)


@pytest.mark.parametrize("status,changes", [
    (-1, dict(x=None)), (-1, dict(codes=None)), (-1, dict(scales=None)), (-1, dict(E=0)),
    (-1, dict(R=0)), (-1, dict(K=0)), (-1, dict(K=-32)), (-1, dict(tr=2)), (-1, dict(tr=-1)),
    (-5, dict(xd=3)), (-5, dict(xd=-1)), (-2, dict(K=48)), (-2, dict(tr=1, R=48)),
    (-7, dict(R=1 << 40)), (-7, dict(E=1 << 42)), (-7, dict(R=1 << 20, K=1 << 21)),
    (-7, dict(tr=1, E=65536)), (-7, dict(tr=1, R=(1 << 23) + 32)),
    (-7, dict(tr=1, K=(1 << 28) + 1)),
    (-1, dict(x=at(0) + 8)), (-1, dict(codes=at(1) + 8)), (-1, dict(tr=1, x=at(0) + 1)),
    (-1, dict(tr=1, xd=0, x=at(0) + 2)), (-1, dict(codes=at(0))), (-1, dict(codes=at(2))),
    (-1, dict(scales=at(0)))])
def test_quantize_refuses(lib, status, changes):
    refuse(lib, status, lib.mxfp4_quantize, QUANT, changes)


DEQUANT = dict(codes=at(0), scales=at(1), R=3, K=64, out=at(2), od=1, stream=None)


@pytest.mark.parametrize("status,changes", [
    (-1, dict(codes=None)), (-1, dict(scales=None)), (-1, dict(out=None)), (-1, dict(R=0)),
    (-1, dict(K=0)), (-2, dict(K=16)), (-5, dict(od=3)), (-7, dict(R=1 << 40)),
    (-1, dict(codes=at(0) + 4)), (-1, dict(out=at(2) + 8)), (-1, dict(out=at(0))),
    (-1, dict(out=at(1)))])
def test_dequantize_refuses(lib, status, changes):
    refuse(lib, status, lib.mxfp4_dequantize, DEQUANT, changes)


GEMM = dict(a=at(0), ad=3, sa=at(1), rows=8, gather=at(2), div=2, blocks=at(3), scales=at(4),
            off=at(5), E=4, P=16, N=64, K=96, epi=0, rs=at(6), scatter=at(7), out=at(8), od=1,
            out_rows=16, ws=None, wsb=0, stream=None)
WIDE = dict(ad=1, sa=None, P=256, out_rows=256, ws=at(9), wsb=1 << 16)


@pytest.mark.parametrize("status,changes", [
    (-1, dict(E=0)), (-2, dict(E=1025)), (-1, dict(P=-1)), (-1, dict(rows=-1)),
    (-1, dict(out_rows=-1)), (-1, dict(N=8)), (-2, dict(N=24)), (-1, dict(K=0)), (-2, dict(K=80)),
    (-1, dict(epi=2)), (-2, dict(epi=1, N=48)), (-5, dict(ad=4)), (-5, dict(ad=-1)),
    (-5, dict(od=3)), (-1, dict(div=0)), (-7, dict(P=(1 << 31) - 1)), (-7, dict(rows=1 << 31)),
    (-7, dict(out_rows=1 << 31)), (-7, dict(rows=1 << 30)), (-7, dict(N=1 << 27)),
    (-7, dict(K=1 << 31)), (-1, dict(a=None)), (-1, dict(blocks=None)), (-1, dict(scales=None)),
    (-1, dict(off=None)), (-1, dict(out=None)), (-1, dict(rows=0)), (-1, dict(out_rows=0)),
    (-1, dict(sa=None)), (-1, dict(ad=1)), (-1, dict(gather=None)), (-1, dict(a=at(0) + 8)),
    (-1, dict(blocks=at(3) + 8)), (-1, dict(out=at(8) + 8)), (-1, dict(gather=at(2) + 2)),
    (-1, dict(off=at(5) + 1)), (-1, dict(rs=at(6) + 2)), (-1, dict(scatter=at(7) + 2)),
    (-6, dict(WIDE, ws=None)), (-6, dict(WIDE, wsb=511)), (-1, dict(WIDE, ws=at(9) + 128))])
def test_product_refuses(lib, status, changes):
    refuse(lib, status, lib.grouped_mx4_gemm, GEMM, changes)


@pytest.mark.parametrize("changes", [dict(P=(1 << 30) - 1, N=1 << 22), dict(P=1 << 24, N=1 << 23, K=32, E=1),
                                     dict(P=1 << 27, N=1 << 17, epi=1)])
def test_product_tiles_are_counted_in_32_bits(lib, changes):
    """Many rows scattered into few places: every array is small, the tiles are not."""
    refuse(lib, -7, lib.grouped_mx4_gemm, GEMM, changes)


@pytest.mark.parametrize("other", ["a", "sa", "gather", "blocks", "scales", "off", "rs", "scatter"])
def test_product_output_is_no_input(lib, other):
    refuse(lib, -1, lib.grouped_mx4_gemm, GEMM, dict(out=GEMM[other]))


@pytest.mark.parametrize("other", ["a", "gather", "blocks", "scales", "off", "rs", "scatter", "out"])
def test_product_workspace_is_no_array(lib, other):
    refuse(lib, -1, lib.grouped_mx4_gemm, GEMM, dict(WIDE, ws=GEMM[other]))


def test_product_of_no_rows(lib):
    args = dict(GEMM, P=0, rows=0, out_rows=0, a=None, out=None)
    assert lib.grouped_mx4_gemm(*args.values()) == 0


def test_product_workspace(lib):
    args = dict(rows=64, ad=1, E=4, P=256, N=64, K=96, epi=0)
    f = lambda **kw: lib.grouped_mx4_gemm_workspace(*dict(args, **kw).values())  # noqa: E731
    assert f() >= 64 * 48 + 64 * 3 and f(ad=0, rows=1 << 20, K=4096) >= (1 << 20) * (2048 + 128)
    assert f(P=8) == 0  # few rows: made in the product's launch
    assert f(P=32, N=1 << 20) > 0
    for bad in (dict(ad=3), dict(rows=0), dict(K=80), dict(K=0), dict(rows=-1), dict(ad=7),
                dict(P=0), dict(E=0), dict(N=0), dict(rows=1 << 40)):
        assert f(**bad) == 0, bad


DISP = dict(x=at(0), xd=1, pos=at(1), w=at(2), T=4, k=2, R=8, H=64, rows=at(3), rd=2, stream=None)
COMB = dict(rows=at(0), rd=1, pos=at(1), w=at(2), T=4, k=2, R=8, H=64, y=at(3), yd=2, stream=None)
BWD = dict(dy=at(0), dyd=1, rows=at(1), rd=2, pos=at(2), w=at(3), T=4, k=2, R=8, H=64,
           drows=at(4), dd=2, dw=at(5), stream=None)
SIZES = [(-1, dict(T=0)), (-4, dict(k=0)), (-4, dict(k=33)), (-1, dict(R=-1)), (-1, dict(H=0)),
         (-2, dict(H=60)), (-7, dict(T=1 << 30)), (-7, dict(R=1 << 31)), (-7, dict(H=1 << 25)),
         (-1, dict(pos=None)), (-1, dict(pos=at(30) + 2)), (-1, dict(w=at(30) + 2))]


@pytest.mark.parametrize("status,changes", SIZES + [
    (-1, dict(x=None)), (-1, dict(rows=None)), (-5, dict(xd=3)), (-5, dict(rd=-1)),
    (-1, dict(x=at(0) + 8)), (-1, dict(rows=at(3) + 8)), (-1, dict(rows=at(0))),
    (-1, dict(rows=at(1))), (-1, dict(rows=at(2)))])
def test_dispatch_refuses(lib, status, changes):
    refuse(lib, status, lib.moe_dispatch, DISP, changes)


@pytest.mark.parametrize("status,changes", SIZES + [
    (-1, dict(rows=None)), (-1, dict(y=None)), (-5, dict(rd=3)), (-5, dict(yd=-1)),
    (-1, dict(rows=at(0) + 8)), (-1, dict(y=at(3) + 8)), (-1, dict(y=at(0))), (-1, dict(y=at(1))),
    (-1, dict(y=at(2)))])
def test_combine_refuses(lib, status, changes):
    refuse(lib, status, lib.moe_combine, COMB, changes)


@pytest.mark.parametrize("status,changes", SIZES + [
    (-1, dict(dy=None)), (-1, dict(rows=None)), (-1, dict(dw=None)), (-5, dict(dyd=3)),
    (-5, dict(rd=3)), (-5, dict(dd=3)), (-1, dict(dy=at(0) + 8)), (-1, dict(rows=at(1) + 8)),
    (-1, dict(drows=at(4) + 8)), (-1, dict(dw=at(5) + 2)), (-1, dict(drows=at(0))),
    (-1, dict(drows=at(2))), (-1, dict(drows=at(3))), (-1, dict(drows=at(5))),
    (-1, dict(drows=at(1), dd=1)), (-1, dict(dw=at(0))), (-1, dict(dw=at(1))),
    (-1, dict(dw=at(2))), (-1, dict(dw=at(3)))])
def test_combine_backward_refuses(lib, status, changes):
    refuse(lib, status, lib.moe_combine_backward, BWD, changes)


def test_dispatch_of_no_rows(lib):
    assert lib.moe_dispatch(*dict(DISP, R=0, rows=None).values()) == 0


ROUTE = dict(logits=at(0), ids=at(1), dw=at(2), T=4, E=8, k=2, renorm=1, dl=at(3), stream=None)


@pytest.mark.parametrize("status,changes", [
    (-1, dict(logits=None)), (-1, dict(ids=None)), (-1, dict(dw=None)), (-1, dict(dl=None)),
    (-1, dict(T=0)), (-1, dict(E=0)), (-2, dict(E=1025)), (-4, dict(k=0)), (-4, dict(k=9)),
    (-7, dict(T=1 << 30)), (-1, dict(renorm=2)), (-1, dict(dl=at(0))), (-1, dict(dl=at(1))),
    (-1, dict(dl=at(2))), (-1, dict(logits=at(0) + 2)), (-1, dict(ids=at(1) + 2)),
    (-1, dict(dw=at(2) + 2)), (-1, dict(dl=at(3) + 2))])
def test_route_backward_refuses(lib, status, changes):
    refuse(lib, status, lib.moe_route_backward, ROUTE, changes)
