"""The block norms' gradients where each workgroup takes rows in several turns, the last of
them cut: the next row's reads, the sums carried over rows and the weights kept for
them, for every number of waves a row.  Oracle and tolerances of test_gpu_blocknorm."""

import pytest

from test_gpu_blocknorm import both, make

pytestmark = pytest.mark.gpu

# rows that one workgroup takes at a time, at most, up to a row length
ROWS = [(512, 16), (1024, 8), (2048, 4), (4096, 2), (16384, 1)]


def several_turns(lib, T, H):
    """The partial rows of the workspace are one a workgroup."""
    groups = lib.load().block_norm_backward_workspace(T, H) // (12 * H)
    rows = next(r for top, r in ROWS if H <= top)
    # at least two turns, and not all of the last one's rows
    return T > groups * rows and T % (groups * rows) != 0


SIZES = [(4099, 264), (2051, 1000), (1029, 2048), (517, 2888), (1031, 4096), (771, 5120), (530, 8208)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_sizes(gpu_lib, T, H, gate, t):
    assert several_turns(gpu_lib, T, H)
    both(gpu_lib, make(T, H, res=t, y=t, h=t, gate=gate), T, H, res=t, y=t, h=t, gate=gate)


@pytest.mark.parametrize("T,H", [(1030, 1544), (519, 2880), (301, 13808)])
@pytest.mark.parametrize("gate", ["token", "channel"])
@pytest.mark.parametrize("res,y,h,w", [("f32", "bf16", "bf16", "bf16"), ("bf16", "f32", "f16", "f32"),
                                       ("f16", "f16", "f32", "f16")])
def test_types(gpu_lib, T, H, gate, res, y, h, w):
    assert several_turns(gpu_lib, T, H)
    both(gpu_lib, make(T, H, res=res, y=y, h=h, w=w, gate=gate), T, H, res=res, y=y, h=h, gate=gate)


@pytest.mark.parametrize("T,H", [(2060, 520), (1030, 1032), (515, 4096), (261, 8200)])
@pytest.mark.parametrize("post,pre,d_r", [(False, True, False), (True, False, True),
                                          (False, False, True)])
def test_parts(gpu_lib, T, H, post, pre, d_r):
    assert several_turns(gpu_lib, T, H)
    both(gpu_lib, make(T, H, post=post, pre=pre, d_r=d_r), T, H)


@pytest.mark.parametrize("T,H", [(4099, 128), (1030, 2048), (261, 8200)])
def test_norm_alone(gpu_lib, T, H):
    """No y: the plain norm's gradient."""
    assert several_turns(gpu_lib, T, H)
    both(gpu_lib, make(T, H, y=None, post=False, gate="none"), T, H, gate="none", beta=1.0)
