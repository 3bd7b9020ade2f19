"""Calls of the operators around the routed experts that their contracts allow: from
several host threads, in place, with every copy of the weights."""

import threading

import numpy as np
import pytest
import torch

import oracle
import test_gpu_blocknorm as norm
import test_gpu_matvec as mv
from oracle import muon
from parity import half_spacing

pytestmark = pytest.mark.gpu
DEV = "cuda"
C = (3.4445, -4.7750, 2.0315)


def host(t):
    return t.detach().double().cpu().numpy()


def randn(*shape, seed=0):
    return torch.randn(*shape, device=DEV, generator=torch.Generator(DEV).manual_seed(seed))


def test_orthogonalize_from_two_threads(gpu_lib):
    """Factors that need different amounts of LDS, whose limit is one per kernel."""
    us = [randn(256, 16, n, seed=n) for n in (700, 2048)]
    want = [gpu_lib.lora_orthogonalize(u) for u in us]
    for u, o in zip(us, want):
        ref = muon.newton_schulz(host(u[:4]), 5, C, 1e-7)
        assert np.all(np.abs(host(o[:4]) - ref) <= half_spacing(ref, "f32") + 1e-9)
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def calls(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(40):
                    got[i].append(gpu_lib.lora_orthogonalize(us[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        assert len(got[i]) == 40 and all(torch.equal(o, want[i]) for o in got[i])


@pytest.mark.parametrize("shape,rank_major", [((130, 8, 256), True), ((130, 256, 8), False),
                                              ((2, 16, 4096), True), ((2, 6001, 7), False)])
@pytest.mark.parametrize("wt,ct", [(torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16),
                                   (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16)])
def test_the_16_bit_copy_is_the_stored_weight_rounded(gpu_lib, shape, rank_major, wt, ct):
    """One workgroup a factor and two launches, aligned and not."""
    w = (0.05 * randn(*shape, seed=1)).to(wt)
    copy = torch.zeros(shape, dtype=ct, device=DEV)
    gpu_lib.lora_muon_step([dict(grad=randn(*shape, seed=2), momentum=randn(*shape, seed=3), w=w,
                                 w16=copy, rank_major=rank_major)], lr=0.3)
    assert torch.equal(copy, w.to(ct))


@pytest.mark.parametrize("T,H", [(4099, 264), (70, 640), (1030, 2048), (517, 2888), (300, 5120),
                                 (261, 8200)])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("dy", ["y", "dh"])
def test_norm_gradients_in_place(gpu_lib, T, H, gate, t, dy):
    """dresidual in d_r_out's place, dy in y's or dh's: the same bits."""
    c = norm.make(T, H, res=t, y=t, h=t, gate=gate)
    kw = dict(w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"], gate_axis=gate, alpha=0.5)
    r = c["residual"]
    want = gpu_lib.block_norm_backward(c["dh"], c["d_r"], r, y=c["y"], **kw)
    place = c["y"] if dy == "y" else c["dh"]
    got = gpu_lib.block_norm_backward(c["dh"], c["d_r"], r, y=c["y"], dresidual=c["d_r"], dy=place,
                                      **kw)
    assert got["dresidual"] is c["d_r"] and got["dy"] is place
    assert set(got) == set(want) and all(torch.equal(got[k], want[k]) for k in want)


def test_norm_gradient_places_are_checked(gpu_lib):
    c = norm.make(4, 64)
    kw = dict(y=c["y"], w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"])
    for bad in (dict(dresidual=c["d_r"][:2]), dict(dy=c["y"].cpu()), dict(dy=c["y"][:, :32]),
                dict(y=None, w_post=None, gate=None, dy=c["y"])):
        with pytest.raises(ValueError):
            gpu_lib.block_norm_backward(c["dh"], c["d_r"], c["residual"], **dict(kw, **bad))
    with pytest.raises(TypeError):
        gpu_lib.block_norm_backward(c["dh"], c["d_r"], c["residual"], dy=c["y"].float(), **kw)
    for bad in (dict(dresidual=c["residual"]), dict(dresidual=c["y"]), dict(dy=c["d_r"])):
        with pytest.raises(gpu_lib.Nf4MoeError):
            gpu_lib.block_norm_backward(c["dh"], c["d_r"], c["residual"], **kw, **bad)


@pytest.mark.parametrize("shape,rank_major", [((2, 16, 4096), True), ((2, 2560, 16), False),
                                              ((2, 6001, 7), False), ((1, 1, 70000), True),
                                              ((3, 16, 3333), True), ((130, 8, 256), True)])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_orthogonalize_in_place(gpu_lib, shape, rank_major, t):
    """Beyond what one workgroup holds too, aligned and not."""
    u = randn(*shape, seed=4).to(t)
    want = gpu_lib.lora_orthogonalize(u, rank_major=rank_major)
    assert gpu_lib.lora_orthogonalize(u, rank_major=rank_major, out=u) is u
    assert torch.equal(u, want)


@pytest.mark.parametrize("T", [38, 48, 63, 64, 65, 130])
@pytest.mark.parametrize("qt,group", [("nf4", 64), ("int4", 128), ("mxfp4", 32)])
@pytest.mark.parametrize("N,K", [(100, 1152), (2500, 192), (70, 4416)])
def test_many_rows_of_x(gpu_lib, T, qt, group, N, K):
    K = K // group * group
    x, codes, st, s, z = mv.make(qt, group, T, N, K)
    ref, mag = oracle.matvec(x.float().numpy(), codes, s, qt, group, z)
    mv.check(mv.run(gpu_lib, x, codes, st, z, qt, group, out_dtype=torch.float32), ref, mag, K, "f32")


@pytest.mark.parametrize("power", [-100, -40, -20, 20, 100])
@pytest.mark.parametrize("T,K", [(1, 256), (5, 256), (16, 2112), (3, 4416), (20, 6208)])
@pytest.mark.parametrize("qt,group", [("fp4", 64), ("mxfp4", 32)])
def test_bf16_rows_of_any_size(gpu_lib, qt, group, T, K, power):
    """The values of fp4 and MXFP4 are bf16 numbers: x keeps its range and its bits."""
    K = K // group * group
    x, codes, st, s, z = mv.make(qt, group, T, 70, K)
    x[:, ::7] *= 2.0 ** -20  # beside values a million times as large
    x = x * 2.0 ** power
    ref, mag = oracle.matvec(x.double().numpy(), codes, s, qt, group)
    mv.check(mv.run(gpu_lib, x, codes, st, z, qt, group, out_dtype=torch.float32), ref, mag, K, "f32")
