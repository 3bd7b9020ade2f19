"""The orthogonalised adapter update on the GPU against 64 bits.

Tolerances: lora_orthogonalize computes in 64 bits from u as given, so O is off by
its own rounding (and 1e-9).  In the optimiser step m' has two roundings of 2^-24 of its
terms, and u one more of its largest element; with |X_0| = 1 an error d of X_0 becomes at
most a^steps d = 485 d in O (a = 3.4445, the steepest slope of the polynomial, at zero).
"""

import numpy as np
import pytest
import torch

from oracle import muon
from parity import half_spacing

pytestmark = pytest.mark.gpu
DEV = "cuda"
TT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
C = (3.4445, -4.7750, 2.0315)
U = 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def factor(E, r, n, rank_major, seed=0):
    """Singular values over four decades, experts of very different sizes."""
    rng = np.random.default_rng((seed, E, r, n))
    u = rng.standard_normal((E, r, r)) @ (np.logspace(0, -4, r)[None, :, None] *
                                          rng.standard_normal((E, r, n)))
    u = u * 10.0 ** rng.uniform(-6, 6, (E, 1, 1))
    u = u if rank_major else u.transpose(0, 2, 1)
    return np.ascontiguousarray(u, dtype=np.float32)


def ns(u, rank_major, steps=5, eps=1e-7):
    return muon.newton_schulz(u, steps, C, eps)


@pytest.mark.parametrize("rank_major", [True, False])
@pytest.mark.parametrize("E,r,n", [(1, 1, 1), (2, 1, 700), (3, 2, 65), (1, 3, 1000), (2, 5, 257),
                                   (4, 7, 31), (3, 8, 2048), (2, 9, 513), (1, 12, 64),
                                   (2, 16, 4100), (5, 16, 16), (2, 16, 5), (1, 11, 3),
                                   (2, 3, 20001), (2, 6, 9000), (3, 16, 3333), (1, 1, 70000),
                                   (260, 16, 2200)])
def test_orthogonalize(gpu_lib, E, r, n, rank_major):
    u = factor(E, r, n, rank_major)
    o = gpu_lib.lora_orthogonalize(torch.from_numpy(u).to(DEV), rank_major=rank_major)
    ref = ns(u, rank_major)
    assert np.all(np.abs(host(o) - ref) <= half_spacing(ref, "f32") + 1e-9)


@pytest.mark.parametrize("rank_major", [True, False])
@pytest.mark.parametrize("r,n", [(1, 1), (1, 30), (2, 33), (3, 50), (4, 64), (5, 1), (6, 129),
                                 (7, 2), (8, 2048), (9, 31), (10, 256), (12, 500), (16, 2048),
                                 (16, 2109), (16, 9), (13, 1024), (4, 8444), (8, 4224)])
def test_orthogonalize_many_factors(gpu_lib, r, n, rank_major):
    """More factors than compute units, below and beyond what one workgroup holds."""
    E = 300
    u = np.concatenate([factor(4, r, n, rank_major, k) for k in range(3)] * 25)
    o = host(gpu_lib.lora_orthogonalize(torch.from_numpy(u).to(DEV), rank_major=rank_major))
    ref = ns(u[:12], rank_major)
    for k in range(0, E, 12):
        assert np.all(np.abs(o[k:k + 12] - ref) <= half_spacing(ref, "f32") + 1e-9), k


@pytest.mark.parametrize("ut", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ot", ["f32", "bf16", "f16"])
def test_orthogonalize_types_in_place_and_steps(gpu_lib, ut, ot):
    u = torch.from_numpy(factor(3, 8, 300, True) * 1e-3).clamp(-1e4, 1e4).to(TT[ut]).to(DEV)
    for steps in (1, 3, 10):
        ref = ns(host(u), True, steps)
        o = gpu_lib.lora_orthogonalize(u, steps=steps, out_dtype=TT[ot])
        assert np.all(np.abs(host(o) - ref) <= 1.001 * half_spacing(ref, ot) + 1e-9 * 4.0 ** steps)
    if ut == ot:
        v = u.clone()
        assert gpu_lib.lora_orthogonalize(v, steps=10, out=v) is v and torch.equal(v, o)


def test_zero_and_non_finite_factors_stay_alone(gpu_lib):
    for rank_major in (True, False):
        u = factor(5, 8, 200, rank_major)
        u[1] = 0
        u[2, 0, 0], u[3, 0, 0] = np.nan, np.inf
        o = host(gpu_lib.lora_orthogonalize(torch.from_numpy(u).to(DEV), rank_major=rank_major))
        assert not o[1].any() and np.isnan(o[2]).all() and np.isnan(o[3]).all()
        ref = ns(u[[0, 4]], rank_major)
        assert np.all(np.abs(o[[0, 4]] - ref) <= half_spacing(ref, "f32") + 1e-9)
    z = torch.zeros(2, 4, 10, device=DEV)
    assert torch.count_nonzero(gpu_lib.lora_orthogonalize(z, eps=0.0)) == 0


def step_case(shapes, wt, seed=0):
    out = []
    for i, (E, r, n, rank_major) in enumerate(shapes):
        rng = np.random.default_rng((seed, i))
        g = factor(E, r, n, rank_major, seed + i)
        m = factor(E, r, n, rank_major, seed + 50 + i)
        w = rng.standard_normal(g.shape).astype(np.float32) * 0.05
        d = dict(grad=torch.from_numpy(g).to(DEV), momentum=torch.from_numpy(m).to(DEV),
                 w=torch.from_numpy(w).to(TT[wt]).to(DEV), rank_major=rank_major, scale=0.2 + i)
        if wt == "f32":
            d["w16"] = torch.empty(d["w"].shape, dtype=(torch.bfloat16, torch.float16)[i % 2],
                                   device=DEV)
        out.append(d)
    return out


def check_step(before, after, wt, lr, mu, nesterov, wd):
    for b, a in zip(before, after):
        g, m0 = host(b["grad"]), host(b["momentum"])
        m = muon.muon_momentum(g, m0, float(np.float32(mu)))
        got = host(a["momentum"])
        assert np.all(np.abs(got - m) <= 2 * U * (np.abs(mu * m0) + np.abs(g)) + 1e-37)
        u = g + float(np.float32(mu)) * got if nesterov else got
        o = ns(u, b["rank_major"])
        w = muon.muon_weight(host(b["w"]), o, lr, wd, b["scale"])
        off = lr * b["scale"] * 485 * U  # u's rounding: at most 2^-24 of |u|, in all
        tol = off + 2 * U * np.abs(w)
        d = np.abs(host(a["w"]) - w)
        assert np.all(d <= tol + half_spacing(w, wt)), (d / (tol + half_spacing(w, wt))).max()
        if wt == "f32":
            kind = "bf16" if a["w16"].dtype == torch.bfloat16 else "f16"
            assert torch.equal(a["w16"], a["w"].to(a["w16"].dtype)), kind


SHAPES = [(4, 8, 2048, True), (4, 8, 1024, False), (3, 5, 100, True), (2, 16, 777, False),
          (1, 1, 9, True), (2, 3, 64, False), (6, 7, 256, True), (1, 16, 2048, True)]


MANY = [(130, 8, 256, True), (130, 8, 256, False), (20, 5, 77, True), (30, 6, 51, False)]
# factors beyond one workgroup, aligned and not
BIG = [(2, 16, 4096, True), (2, 16, 2560, False), (1, 8, 8192, False), (3, 4, 512, True)]
BIG_ODD = [(2, 16, 4099, True), (2, 7, 6001, False)]


@pytest.mark.parametrize("wt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shapes", [SHAPES[:1], SHAPES[:4], SHAPES, MANY, BIG, BIG_ODD])
def test_step(gpu_lib, wt, nesterov, shapes):
    t = step_case(shapes, wt)
    before = [{k: v.clone() if torch.is_tensor(v) else v for k, v in d.items()} for d in t]
    gpu_lib.lora_muon_step(t, lr=0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1)
    check_step(before, t, wt, 0.02, 0.9, nesterov, 0.1)
    for b, a in zip(before, t):
        assert torch.equal(b["grad"], a["grad"])


@pytest.mark.parametrize("shapes", [SHAPES[:4], MANY])
def test_step_out_of_place_is_in_place_and_repeats(gpu_lib, shapes):
    t = step_case(shapes, "bf16")
    out = [dict(d, momentum_out=torch.empty_like(d["momentum"]), w_out=torch.empty_like(d["w"]))
           for d in t]
    kept = [(d["momentum"].clone(), d["w"].clone()) for d in t]
    for _ in range(2):
        gpu_lib.lora_muon_step(out, lr=0.1)
    assert all(torch.equal(d["momentum"], m) and torch.equal(d["w"], w) for d, (m, w) in zip(t, kept))
    gpu_lib.lora_muon_step(t, lr=0.1)
    for d, o in zip(t, out):
        assert torch.equal(d["momentum"], o["momentum_out"]) and torch.equal(d["w"], o["w_out"])


def test_step_graph_replays_carry_the_state(gpu_lib):
    """Each replay is one more step, as eager calls on another stream make them."""
    a, b = step_case(SHAPES[:2], "f32"), step_case(SHAPES[:2], "f32")
    kw = dict(lr=0.05, momentum=0.8, weight_decay=0.01)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpu_lib.lora_muon_step(a, **kw)
        gpu_lib.lora_muon_step(b, **kw)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.lora_muon_step(a, **kw)
    for i in range(3):
        for x, y in zip(a, b):
            x["grad"].mul_(-0.5)
            y["grad"].mul_(-0.5)
        g.replay()
        torch.cuda.synchronize()
        gpu_lib.lora_muon_step(b, **kw)
        for x, y in zip(a, b):
            assert torch.equal(x["w"], y["w"]) and torch.equal(x["momentum"], y["momentum"])
            assert torch.equal(x["w16"], y["w16"])


def test_binding_refuses_on_the_gpu(gpu_lib):
    t = step_case(SHAPES[:1], "f32")[0]
    for bad in (dict(momentum=t["momentum"][:2]), dict(grad=t["grad"].cpu()),
                dict(w=t["w"][:, :, :64].contiguous()), dict(grad=t["grad"][0])):
        with pytest.raises(ValueError):
            gpu_lib.lora_muon_step([dict(t, **bad)], lr=0.1)
    with pytest.raises(TypeError):
        gpu_lib.lora_muon_step([dict(t, momentum=t["momentum"].half())], lr=0.1)
    with pytest.raises(gpu_lib.Nf4MoeError):
        gpu_lib.lora_muon_step([t], lr=float("nan"))
    with pytest.raises(gpu_lib.Nf4MoeError):
        gpu_lib.lora_orthogonalize(torch.zeros(1, 17, 64, device=DEV))
