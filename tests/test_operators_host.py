"""Refusals of the operators around the routed experts: every bad argument is
found on the host, before anything is enqueued (CPU only, no kernel runs)."""

import ctypes

import pytest

from grouped_nf4_gemm_quantize_amd import binding

FAKE = 0x10000  # a 64 KiB-aligned non-null pointer; never dereferenced here
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def _refuse(lib, status, fn, defaults, changes):
    args = dict(defaults, **changes)
    assert fn(*args.values()) == status, (changes, lib.nf4moe_last_error())
    assert lib.nf4moe_last_error()


MATVEC = dict(qt=0, x=FAKE, xd=2, T=1, codes=FAKE, scales=FAKE, sd=0, zeros=None, group=64, N=5,
              K=128, bias=None, y=FAKE + 0x1000, yd=1, stream=None)


@pytest.mark.parametrize("status,changes", [
    (-1, dict(qt=3)), (-1, dict(qt=-1)), (-1, dict(qt=5)), (-1, dict(x=None)),
    (-1, dict(codes=None)), (-1, dict(scales=None)), (-1, dict(y=None)), (-1, dict(T=0)),
    (-1, dict(N=0)), (-1, dict(K=0)), (-1, dict(T=-4)), (-5, dict(xd=0)), (-5, dict(xd=9)),
    (-5, dict(yd=3)), (-3, dict(group=32)), (-3, dict(group=128)), (-3, dict(qt=2, group=16)),
    (-3, dict(qt=7)), (-1, dict(zeros=FAKE)), (-1, dict(qt=7, group=32, zeros=FAKE)),
    (-5, dict(sd=1)), (-5, dict(qt=2, sd=7)), (-2, dict(K=96)), (-2, dict(qt=7, group=32, K=48)),
    (-2, dict(qt=2, group=128, K=192)), (-7, dict(T=262145)), (-7, dict(N=1 << 31)),
    (-7, dict(K=(1 << 24) + 64)), (-1, dict(x=FAKE + 8)), (-1, dict(codes=FAKE + 4)),
    (-1, dict(y=FAKE)), (-1, dict(scales=FAKE + 2)), (-1, dict(bias=FAKE + 2)), (-1, dict(y=FAKE + 1)),
    (-1, dict(qt=2, sd=2, scales=FAKE + 1))])
def test_matvec_refuses(lib, status, changes):
    _refuse(lib, status, lib.nbit_matvec, MATVEC, changes)


B, C, D, F = (FAKE + 0x1000 * i for i in range(1, 5))  # further arrays
NORM = dict(res=FAKE, rd=1, y=B, yd=1, gate=None, axis=0, w_pre=FAKE, w_post=FAKE, wd=1,
            off=0.0, alpha=1.0, beta=1.0, eps=1e-6, T=4, H=64, r_out=C, h=D, hd=1,
            stream=None)
NORM_SHARED = [
    (-1, dict(T=0)), (-1, dict(H=0)), (-2, dict(H=68)), (-2, dict(H=16392)),
    (-7, dict(T=1 << 31)), (-1, dict(axis=1)), (-1, dict(gate=FAKE)), (-1, dict(gate=FAKE, axis=3)),
    (-5, dict(rd=4)), (-5, dict(yd=-1)), (-5, dict(hd=3)), (-5, dict(wd=3)), (-1, dict(alpha=NAN)),
    (-1, dict(beta=INF)), (-1, dict(off=NAN)), (-1, dict(eps=-1e-6)), (-1, dict(eps=NAN)),
    (-1, dict(y=FAKE + 8)), (-1, dict(w_pre=FAKE + 2)), (-1, dict(w_post=FAKE + 8))]


@pytest.mark.parametrize("status,changes", NORM_SHARED + [
    (-1, dict(res=None)), (-1, dict(r_out=None)), (-1, dict(h=None)),
    (-1, dict(y=None, r_out=None)),                             # w_post without y
    (-1, dict(y=None, r_out=None, w_post=None, beta=0.5)), (-1, dict(y=None, w_post=None)),
    (-1, dict(y=None, r_out=None, w_post=None, w_pre=None, h=None)),
    (-1, dict(y=None, r_out=None, w_post=None, gate=FAKE, axis=1)), (-1, dict(w_pre=None)),
    (-1, dict(res=FAKE + 4)), (-1, dict(r_out=FAKE + 8)), (-1, dict(h=FAKE + 8)),
    (-1, dict(h=C)), (-1, dict(h=FAKE)), (-1, dict(h=B, yd=0)), (-1, dict(r_out=B)),
    (-1, dict(gate=FAKE + 2, axis=1))])
def test_block_norm_refuses(lib, status, changes):
    _refuse(lib, status, lib.block_norm_forward, NORM, changes)


NORM_BWD = dict(dh=FAKE, hd=1, d_r=B, r=C, rd=1, y=D, yd=1, gate=None, axis=0, w_pre=FAKE,
                w_post=FAKE, wd=1, off=0.0, alpha=1.0, beta=1.0, eps=1e-6, T=4, H=64, dres=F,
                dy=F + 0x1000, dgate=None, dw_pre=FAKE, dw_post=FAKE, ws=FAKE, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("status,changes", [
    (s, dict(c, dgate=FAKE) if "gate" in c else c) for s, c in NORM_SHARED] + [
    (-1, dict(r=None)), (-1, dict(dres=None)), (-1, dict(dh=None)), (-1, dict(dy=None)),
    (-1, dict(dw_pre=None)), (-1, dict(dw_post=None)), (-1, dict(dgate=FAKE)),
    (-1, dict(gate=FAKE, axis=1)), (-1, dict(dh=None, d_r=None, w_pre=None, dw_pre=None)),
    (-1, dict(w_post=None)), (-1, dict(dh=FAKE + 8)), (-1, dict(d_r=FAKE + 8)),
    (-1, dict(dres=FAKE + 4)), (-1, dict(dy=FAKE + 4)), (-1, dict(dw_pre=FAKE + 2)),
    (-1, dict(dres=D)), (-1, dict(dres=FAKE)), (-1, dict(dres=C)), (-1, dict(dres=F + 0x1000)),
    (-1, dict(dy=C)), (-1, dict(dy=B)), (-1, dict(dy=FAKE, yd=0)),
    (-1, dict(dw_post=FAKE + 2)), (-6, dict(ws=None)), (-6, dict(wsb=0)), (-1, dict(ws=FAKE + 16))])
def test_block_norm_backward_refuses(lib, status, changes):
    _refuse(lib, status, lib.block_norm_backward, NORM_BWD, changes)


def test_block_norm_backward_workspace_size(lib):
    ws = lib.block_norm_backward_workspace
    assert ws(1, 64) >= 3 * 64 * 4 and ws(1 << 20, 16384) < 1 << 30
    for T, H in ((0, 64), (4, 0), (4, 12), (4, 16392), (1 << 31, 64)):
        assert ws(T, H) == 0
    need = ws(4, 64)
    _refuse(lib, -6, lib.block_norm_backward, NORM_BWD, dict(wsb=need - 1))


def _tensor(**kw):
    d = dict(grad=FAKE, m=B, m_out=B, w=C, w_out=C, w16=None, n=4096, E=2, r=8,
             rank_major=1, w_dtype=0, w16_dtype=0, scale=1.0)
    d.update(kw)
    return binding.MuonTensorStruct(*d.values())


MUON = dict(t=None, count=1, lr=0.1, mu=0.9, nesterov=1, wd=0.0, steps=5, a=3.4, b=-4.7, c=2.0,
            eps=1e-7, ws=FAKE, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("status,tensor,changes", [
    (-1, {}, dict(count=0)), (-1, {}, dict(count=9)), (-1, {}, dict(t=None)),
    (-1, {}, dict(steps=0)), (-1, {}, dict(steps=17)), (-1, {}, dict(a=NAN)),
    (-1, {}, dict(eps=-1.0)), (-1, {}, dict(lr=INF)), (-1, {}, dict(mu=NAN)),
    (-1, {}, dict(wd=NAN)), (-1, {}, dict(nesterov=2)), (-6, {}, dict(ws=None)),
    (-6, {}, dict(wsb=8)), (-1, {}, dict(ws=FAKE + 8)), (-1, dict(grad=None), {}),
    (-1, dict(m=None), {}), (-1, dict(m_out=None), {}), (-1, dict(w=None), {}),
    (-1, dict(w_out=None), {}), (-1, dict(E=0), {}), (-1, dict(n=0), {}), (-1, dict(r=0), {}),
    (-1, dict(r=17), {}), (-1, dict(rank_major=2), {}), (-5, dict(w_dtype=4), {}),
    (-5, dict(w16=FAKE, w16_dtype=0), {}), (-1, dict(scale=NAN), {}), (-1, dict(grad=FAKE + 2), {}),
    (-1, dict(w=FAKE + 2), {}), (-1, dict(w16=FAKE + 1, w16_dtype=1), {}),
    (-7, dict(n=1 << 40), {}), (-7, dict(E=1 << 30), {}), (-7, dict(E=(1 << 18) + 1, n=64), {})])
def test_muon_step_refuses(lib, status, tensor, changes):
    arr = (binding.MuonTensorStruct * 1)(_tensor(**tensor))
    _refuse(lib, status, lib.lora_muon_step, dict(MUON, t=arr), changes)


@pytest.mark.parametrize("first,second", [
    (dict(m_out=FAKE), {}), (dict(w_out=B), {}), (dict(w_out=FAKE), {}), (dict(m_out=C), {}),
    (dict(w16=C, w16_dtype=1), {}), (dict(w16=B, w16_dtype=1), {}), ({}, {}),
    ({}, dict(grad=B, m=D, m_out=D, w=F, w_out=F)), ({}, dict(m=D, m_out=D, w=F, w_out=C)),
    ({}, dict(m=D, m_out=D, w=C, w_out=F)), (dict(w16=D, w16_dtype=1), dict(m=D, m_out=F, w=F + 4096,
                                                                            w_out=F + 4096))])
def test_muon_step_refuses_shared_outputs(lib, first, second):
    """A tensor with itself, or the same array in two tensors."""
    arr = (binding.MuonTensorStruct * 2)(_tensor(**first), _tensor(**second))
    args = dict(MUON, t=arr, count=1 if first and not second else 2)
    _refuse(lib, -1, lib.lora_muon_step, args, {})


def test_muon_workspace_sizes(lib):
    arr = (binding.MuonTensorStruct * 2)(_tensor(), _tensor(r=16, n=2000, E=3))
    one = lib.lora_orthogonalize_workspace(2, 8, 4096)
    assert one >= 2 * 64 * 8
    assert lib.lora_muon_step_workspace(arr, 2) == one + lib.lora_orthogonalize_workspace(3, 16,
                                                                                        2000)
    # small factors need none
    assert lib.lora_orthogonalize_workspace(2, 8, 64) == 0
    assert lib.lora_muon_step_workspace((binding.MuonTensorStruct * 1)(_tensor(n=64)), 1) == 0
    assert lib.lora_muon_step_workspace(arr, 0) == 0 and lib.lora_muon_step_workspace(None, 1) == 0
    assert lib.lora_muon_step_workspace((binding.MuonTensorStruct * 1)(_tensor(r=0)), 1) == 0
    for E, r, n in ((0, 8, 64), (2, 17, 64), (2, 8, 0)):
        assert lib.lora_orthogonalize_workspace(E, r, n) == 0


ORTH = dict(u=FAKE, ud=0, E=2, r=8, n=4096, rm=1, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7, out=B,
            od=0, ws=FAKE, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("status,changes", [
    (-1, dict(u=None)), (-1, dict(out=None)), (-5, dict(ud=3)), (-5, dict(od=-1)),
    (-1, dict(out=FAKE, od=1)), (-1, dict(E=0)), (-1, dict(r=17)), (-1, dict(n=0)), (-1, dict(rm=2)), (-1, dict(steps=0)),
    (-1, dict(c=INF)), (-1, dict(u=FAKE + 2)), (-1, dict(od=1, out=FAKE + 1)),
    (-6, dict(wsb=0)), (-6, dict(ws=None)), (-7, dict(n=1 << 41))])
def test_orthogonalize_refuses(lib, status, changes):
    _refuse(lib, status, lib.lora_orthogonalize, ORTH, changes)


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    import torch

    x = torch.zeros(1, 64, dtype=torch.float16)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="GPU"):
        binding.nbit_matvec(x, codes, scales)
    with pytest.raises(ValueError, match="quant_type"):
        binding.nbit_matvec(x, codes, scales, quant_type="int8")
    with pytest.raises(ValueError, match="multiple of the group"):
        binding.nbit_matvec(x, codes, scales, quant_type="int4", group=48)
    with pytest.raises(ValueError, match="GPU"):
        binding.block_norm(x, w_pre=torch.zeros(64))
    with pytest.raises(ValueError, match="gate_axis"):
        binding.block_norm(x, y=x, gate=torch.zeros(1), gate_axis="row")
    with pytest.raises(ValueError, match="1 to 8"):
        binding.lora_muon_step([], lr=0.1)
    with pytest.raises(ValueError, match="must be"):
        binding.lora_orthogonalize(x)
