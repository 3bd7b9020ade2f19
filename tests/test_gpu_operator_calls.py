"""Calls of the operators around the routed experts that their contracts allow: from
several host threads, in place, with every copy of the weights."""

import threading

import numpy as np
import pytest
import torch

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
