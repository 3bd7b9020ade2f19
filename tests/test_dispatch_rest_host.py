"""Refusals of the type that asks for rows without a pair to become 0 (CPU only)."""

import pytest

from grouped_nf4_gemm_quantize_amd import binding
from test_mx4_dispatch_host import BWD, DISP, at, lib, refuse  # noqa: F401

REST = binding.ZERO_REST


@pytest.mark.parametrize("status,changes", [
    (-5, dict(dd=3 | REST)), (-5, dict(dd=REST << 1)), (-5, dict(dd=2 | REST << 1)),
    (-5, dict(dyd=1 | REST)), (-5, dict(rd=2 | REST)), (-5, dict(dd=-1)),
    (-1, dict(dd=2 | REST, drows=BWD["rows"])), (-1, dict(dd=2 | REST, drows=BWD["dy"])),
    (-1, dict(dd=2 | REST, drows=at(4) + 8)), (-2, dict(dd=2 | REST, H=60))])
def test_combine_backward_refuses(lib, status, changes):  # noqa: F811
    refuse(lib, status, lib.moe_combine_backward, BWD, changes)


@pytest.mark.parametrize("status,changes", [
    (-5, dict(rd=3 | REST)), (-5, dict(rd=REST << 1)), (-5, dict(xd=1 | REST)), (-5, dict(rd=-1)),
    (-1, dict(rd=2 | REST, rows=DISP["x"])), (-1, dict(rd=2 | REST, rows=at(3) + 8)),
    (-1, dict(rd=2 | REST, rows=None)), (-2, dict(rd=2 | REST, H=60))])
def test_dispatch_refuses(lib, status, changes):  # noqa: F811
    refuse(lib, status, lib.moe_dispatch, DISP, changes)


def test_no_rows_to_clear(lib):  # noqa: F811
    assert lib.moe_dispatch(*dict(DISP, R=0, rows=None, rd=2 | REST).values()) == 0
