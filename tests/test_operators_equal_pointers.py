"""Equal pointers of the operators around the routed experts: an output that is another
array of the call is refused on the host (CPU only, no kernel runs)."""

import pytest

from grouped_nf4_gemm_quantize_amd import binding

EINVAL = -1


def at(i):
    return 0x100000 * (i + 1)  # distinct aligned pointers, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def refuse(lib, fn, args, a, b):
    """The call is refused because pointer ``a`` equals pointer ``b``."""
    assert fn(*dict(args, **{a: args[b]}).values()) == EINVAL, (a, b)
    assert lib.nf4moe_last_error()


MATVEC = dict(qt=2, x=at(0), xd=2, T=1, codes=at(1), scales=at(2), sd=0, zeros=at(3), group=64, N=5,
              K=128, bias=at(4), y=at(5), yd=0, stream=None)


@pytest.mark.parametrize("other", ["x", "codes", "scales", "zeros", "bias"])
def test_matvec_output(lib, other):
    refuse(lib, lib.nbit_matvec, MATVEC, "y", other)


NORM = dict(res=at(0), rd=1, y=at(1), yd=1, gate=at(2), axis=1, w_pre=at(3), w_post=at(4), wd=1,
            off=0.0, alpha=1.0, beta=1.0, eps=1e-6, T=4, H=64, r_out=at(5), h=at(6), hd=1, stream=None)


@pytest.mark.parametrize("out,other", [(o, i) for o in ("r_out", "h")
                                       for i in ("y", "res", "gate", "w_pre", "w_post")
                                       if (o, i) not in (("r_out", "res"), ("h", "y"))])
def test_norm_outputs(lib, out, other):
    refuse(lib, lib.block_norm_forward, NORM, out, other)


BWD = dict(dh=at(0), hd=1, d_r=at(1), r=at(2), rd=1, y=at(3), yd=1, gate=at(4), axis=1, w_pre=at(5),
           w_post=at(6), wd=1, off=0.0, alpha=1.0, beta=1.0, eps=1e-6, T=4, H=64, dres=at(7),
           dy=at(8), dgate=at(9), dw_pre=at(10), dw_post=at(11), ws=at(12), wsb=1 << 20, stream=None)
BWD_OUT = ["dres", "dy", "dgate", "dw_pre", "dw_post", "ws"]
BWD_IN = ["dh", "d_r", "r", "y", "gate", "w_pre", "w_post"]
IN_PLACE = {("dres", "d_r"), ("dy", "y"), ("dy", "dh")}


@pytest.mark.parametrize("out,other", [(o, i) for o in BWD_OUT for i in BWD_OUT + BWD_IN
                                       if o != i and (o, i) not in IN_PLACE])
def test_norm_gradients(lib, out, other):
    refuse(lib, lib.block_norm_backward, BWD, out, other)
