"""Dispatch, combine and their gradients on the GPU against 64 bits.

Tolerances: dispatch is one fp32 product and one rounding to the rows' type.  Combine
adds k products: k + 1 roundings of 2^-24 of the terms' magnitudes and the rounding of y.  A dot
product over H adds H terms, in at most H/8 + 16 steps one after another (eight columns of a
lane, then lanes and waves), each 2^-24 of the magnitudes, and the product's own rounding.
The softmax: expf and the division are off by at most 2^-21 of a weight (a few units in the
last place), sums over E by log2(E) + E/64 steps of 2^-24.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import dispatch
from parity import half_spacing

pytestmark = pytest.mark.gpu
DEV = "cuda"
TT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def make(T, k, H, R=None, drop=0.0, seed=0, xt="f32", rt="f32"):
    """x, rows, w and a placement of the pairs; R beyond T*k leaves rows free."""
    rng = np.random.default_rng((seed, T, k, H))
    R = T * k if R is None else R
    pos = np.full(T * k, -1, dtype=np.int32)
    n = min(R, T * k)
    pos[rng.permutation(T * k)[:n]] = rng.permutation(R)[:n]
    if drop:
        pos[rng.random(T * k) < drop] = -1
        pos[rng.random(T * k) < drop / 4] = R  # outside at the other end
        pos[rng.random(T * k) < drop / 4] = 2 ** 31 - 1
    t = lambda a, d: torch.from_numpy(a.astype(np.float32)).to(TT[d]).to(DEV)  # noqa: E731
    return dict(x=t(rng.standard_normal((T, H)), xt), rows=t(rng.standard_normal((R, H)), rt),
                w=torch.from_numpy(rng.random((T, k), dtype=np.float32)).to(DEV),
                pos=torch.from_numpy(pos).to(DEV), T=T, k=k, H=H, R=R)


def close(got, want, tol):
    bad = ~(np.abs(host(got) - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(host(got) - want)[bad][:4])


SHAPES = [(1, 1, 8), (1, 8, 2048), (3, 2, 64), (16, 8, 2048), (33, 4, 2880), (200, 6, 136),
          (5, 32, 1448), (2, 3, 16384), (7, 1, 24), (1000, 2, 8), (21, 9, 512), (13, 17, 520), (6, 31, 504)]
PAIRS = [(a, b) for a in TT for b in TT]


def check_dispatch(lib, c, weighted, ot):
    out = torch.full((c["R"], c["H"]), 7.0, device=DEV, dtype=TT[ot])
    w = c["w"] if weighted else None
    got = lib.moe_dispatch(c["x"], c["pos"], c["k"], w=w, out=out)
    want = dispatch.dispatch(host(c["x"]), host(c["pos"]), c["k"], np.full((c["R"], c["H"]), 7.0),
                             None if w is None else host(w))
    close(got, want, half_spacing(want, ot) + (U * np.abs(want) if weighted else 0))


def check_combine(lib, c, weighted, yt):
    w = c["w"] if weighted else None
    got = lib.moe_combine(c["rows"], c["pos"], c["k"], w=w, y_dtype=TT[yt])
    hw = None if w is None else host(w)
    want = dispatch.combine(host(c["rows"]), host(c["pos"]), c["k"], hw)
    mag = dispatch.combine(np.abs(host(c["rows"])), host(c["pos"]), c["k"], hw)
    close(got, want, half_spacing(want, yt) + (c["k"] + 1) * U * mag)


def check_backward(lib, c, weighted, dt, **kw):
    w = c["w"] if weighted else None
    hw = None if w is None else host(w)
    hx, hr, hp = host(c["x"]), host(c["rows"]), host(c["pos"])
    keep = torch.full((c["R"], c["H"]), 7.0, device=DEV, dtype=TT[dt])
    drows, dw = lib.moe_combine_backward(c["x"], c["rows"], c["pos"], c["k"], w=w,
                                         **(kw or dict(drows=keep)))
    _, want = dispatch.combine_backward(hx, hr, hp, c["k"], hw)
    _, mag = dispatch.combine_backward(np.abs(hx), np.abs(hr), hp, c["k"], hw)
    close(dw, want, (c["H"] / 8 + 17) * U * mag)
    if drows is not None:
        at = hp[(hp >= 0) & (hp < c["R"])].astype(int)
        start = hr if drows is c["rows"] else np.full((c["R"], c["H"]), 7.0)
        want = dispatch.dispatch(hx, hp, c["k"], start, hw)
        close(drows, want, half_spacing(want, dt) + (U * np.abs(want) if weighted else 0))
        assert len(at) <= c["R"]
    return drows, dw


@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_shapes(gpu_lib, T, k, H, weighted):
    c = make(T, k, H, xt="bf16", rt="f16")
    check_dispatch(gpu_lib, c, weighted, "f16")
    check_combine(gpu_lib, c, weighted, "bf16")
    check_backward(gpu_lib, c, weighted, "f16")


@pytest.mark.parametrize("a,b", PAIRS)
def test_types(gpu_lib, a, b):
    for T, k, H in ((9, 3, 264), (4, 8, 2048)):
        c = make(T, k, H, xt=a, rt=b)
        check_dispatch(gpu_lib, c, True, b)
        check_combine(gpu_lib, c, True, a)
        for d in TT:
            check_backward(gpu_lib, c, True, d)


@pytest.mark.parametrize("T,k,H,R", [(40, 4, 72, 100), (40, 4, 72, 200), (11, 8, 1032, 64),
                                     (11, 8, 1032, 1), (300, 2, 16, 777)])
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
def test_dropped_pairs_and_free_rows(gpu_lib, T, k, H, R, drop):
    c = make(T, k, H, R=R, drop=drop)
    for weighted in (False, True):
        check_dispatch(gpu_lib, c, weighted, "f32")
        check_combine(gpu_lib, c, weighted, "f32")
        check_backward(gpu_lib, c, weighted, "f32")


def test_no_rows_at_all(gpu_lib):
    c = make(5, 2, 64, R=3)
    c["pos"].fill_(-1)
    none = torch.empty(0, 64, device=DEV)
    assert gpu_lib.moe_dispatch(c["x"], c["pos"], 2, out=none).shape == (0, 64)
    assert (gpu_lib.moe_combine(none, c["pos"], 2) == 0).all()
    drows, dw = gpu_lib.moe_combine_backward(c["x"], none, c["pos"], 2)
    assert drows.shape == (0, 64) and (dw == 0).all()
    # positions that would be rows, but there are none
    c["pos"].fill_(0)
    assert (gpu_lib.moe_combine(none, c["pos"], 2) == 0).all()


def test_non_finite_rows_reach_their_token_only(gpu_lib):
    c = make(12, 3, 136, drop=0.2, seed=4)
    pos = host(c["pos"]).astype(int)
    p = int(np.flatnonzero((pos >= 0) & (pos < c["R"]))[4])
    c["rows"][pos[p], 5] = float("nan")
    free = np.setdiff1d(np.arange(c["R"]), pos)
    c["rows"][torch.from_numpy(free).to(DEV)] = float("inf")  # rows of dropped pairs
    y = host(gpu_lib.moe_combine(c["rows"], c["pos"], 3, w=c["w"]))
    bad = np.zeros(y.shape, bool)
    bad[p // 3, 5] = True
    assert np.array_equal(~np.isfinite(y), bad)
    _, dw = gpu_lib.moe_combine_backward(c["x"], c["rows"], c["pos"], 3, w=c["w"])
    bad = np.zeros(36, bool)
    bad[p] = True
    assert np.array_equal(~np.isfinite(host(dw).reshape(-1)), bad)


@pytest.mark.parametrize("T,k,H", [(9, 3, 264), (3, 20, 2056), (70, 2, 32)])
def test_gradient_in_the_place_of_the_rows(gpu_lib, T, k, H):
    c = make(T, k, H, drop=0.1)
    first = check_backward(gpu_lib, c, True, "f32", need_drows=False)
    assert first[0] is None
    c2 = dict(c, rows=c["rows"].clone())
    drows, dw = gpu_lib.moe_combine_backward(c["x"], c2["rows"], c["pos"], k, w=c["w"],
                                             drows=c2["rows"])
    want, _ = gpu_lib.moe_combine_backward(c["x"], c["rows"], c["pos"], k, w=c["w"],
                                           drows=c["rows"].clone())
    assert torch.equal(drows, want) and torch.equal(dw, first[1])


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (5, 64, 8), (37, 128, 6), (3, 1024, 32),
                                   (9, 65, 3), (130, 256, 1)])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient(gpu_lib, T, E, k, renorm):
    rng = np.random.default_rng((T, E, k))
    logits = (rng.standard_normal((T, E)) * 3).astype(np.float32)
    r = gpu_lib.route_permute(torch.from_numpy(logits).to(DEV), k, renormalize=renorm)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    got = gpu_lib.moe_route_backward(torch.from_numpy(logits).to(DEV), r["ids"],
                                     torch.from_numpy(dw).to(DEV), renormalize=renorm)
    ids = host(r["ids"]).astype(int)
    want = dispatch.route_backward(logits, ids, dw, renorm)
    w = dispatch.route_weights(logits, ids, renorm)
    p = dispatch.route_weights(logits, np.tile(np.arange(E), (T, 1)), False)
    size = np.abs(dw).max(1, keepdims=True) + (w * np.abs(dw)).sum(1, keepdims=True)
    share = np.zeros((T, E))
    np.put_along_axis(share, ids, w, 1)
    share = share if renorm else p
    steps = 2.0 ** -20 + (np.log2(E) + E / 64 + k) * U * 2
    close(got, want, steps * share * size + 1e-37)


def test_router_gradient_of_masked_experts(gpu_lib):
    """Experts that are ruled out (-inf) and choices that are none."""
    T, E, k = 6, 16, 4
    rng = np.random.default_rng(1)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(-logits, 1)[:, :k].astype(np.int32)
    masked = logits.copy()
    np.put_along_axis(masked, np.argsort(logits, 1)[:, :3], -np.inf, 1)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    for renorm in (False, True):
        got = gpu_lib.moe_route_backward(d(masked), d(ids), d(dw), renormalize=renorm)
        want = dispatch.route_backward(masked, ids, dw, renorm)
        close(got, want, 2.0 ** -19 * np.abs(dw).max())
        assert (host(got)[np.isinf(masked)] == 0).all()
    # a choice outside [0, E): no part in the weights
    ids[2, 1], ids[3, 3] = -1, E
    got = host(gpu_lib.moe_route_backward(d(logits), d(ids), d(dw)))
    for t, j in ((2, 1), (3, 3)):
        keep = np.delete(np.arange(k), j)
        want = dispatch.route_backward(logits[t:t + 1], ids[t:t + 1, keep], dw[t:t + 1, keep])
        assert np.abs(got[t] - want[0]).max() <= 2.0 ** -19 * np.abs(dw).max()


@pytest.mark.parametrize("fill", [-np.inf, np.nan, np.inf, 1.0])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_of_tokens_without_a_choice(gpu_lib, renorm, fill):
    """Padded tokens (no choice in [0, E)) get 0, whatever their logits and dw hold."""
    T, E, k = 9, 80, 4
    rng = np.random.default_rng(2)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(-logits, 1)[:, :k].astype(np.int32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    none = [1, 4, 8]
    ids[none], logits[none], dw[none] = (-1, E, -7, 2 ** 31 - 1), fill, np.nan
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    got = host(gpu_lib.moe_route_backward(d(logits), d(ids), d(dw), renormalize=renorm))
    assert (got[none] == 0).all()
    rest = np.setdiff1d(np.arange(T), none)
    want = dispatch.route_backward(logits[rest], ids[rest], dw[rest], renorm)
    assert np.abs(got[rest] - want).max() <= 2.0 ** -19 * np.abs(dw[rest]).max()


def test_captured_and_replayed(gpu_lib):
    c = make(50, 4, 264, drop=0.1)
    out = torch.zeros(c["R"], c["H"], device=DEV)
    y = torch.empty(50, 264, device=DEV)
    dr = torch.zeros(c["R"], c["H"], device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.moe_dispatch(c["x"], c["pos"], 4, w=c["w"], out=out)
        gpu_lib.moe_combine(out, c["pos"], 4, w=c["w"], y=y)
        _, dw = gpu_lib.moe_combine_backward(y, out, c["pos"], 4, w=c["w"], drows=dr)
    for i in range(3):
        c["x"].copy_(torch.randn_like(c["x"]))
        graph.replay()
        torch.cuda.synchronize()
        o = gpu_lib.moe_dispatch(c["x"], c["pos"], 4, w=c["w"], out=torch.zeros_like(out))
        y2 = gpu_lib.moe_combine(o, c["pos"], 4, w=c["w"])
        d2, dw2 = gpu_lib.moe_combine_backward(y2, o, c["pos"], 4, w=c["w"],
                                               drows=torch.zeros_like(dr))
        assert torch.equal(o, out) and torch.equal(y, y2) and torch.equal(dr, d2)
        assert torch.equal(dw, dw2)


def test_on_another_stream(gpu_lib):
    c = make(64, 4, 512, xt="bf16", rt="bf16")
    want = gpu_lib.moe_dispatch(c["x"], c["pos"], 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = c["x"] * 1  # made on this stream
        got = gpu_lib.moe_dispatch(x, c["pos"], 4)
        y = gpu_lib.moe_combine(got, c["pos"].view(64, 4), 4)
    s.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(y, gpu_lib.moe_combine(want, c["pos"], 4))


def test_refusals_of_the_binding(gpu_lib):
    c = make(6, 2, 64)
    x, pos, w, rows = c["x"], c["pos"], c["w"], c["rows"]
    f, g, h = gpu_lib.moe_dispatch, gpu_lib.moe_combine, gpu_lib.moe_combine_backward
    for bad in (lambda: f(x, pos[:11], 2), lambda: f(x, pos.view(4, 3), 2), lambda: f(x[0], pos, 2),
                lambda: f(x, pos, 2, w=w[:5]), lambda: f(x, pos.cpu(), 2),
                lambda: f(x, pos, 2, out=torch.empty(12, 63, device=DEV)),
                lambda: f(x.t(), pos, 2), lambda: g(rows, pos, 5), lambda: g(rows, pos, 0),
                lambda: g(rows, pos, 2, y=x[:5]), lambda: h(x, rows[:, :56], pos, 2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(x, pos.long(), 2), lambda: f(x, pos, 2, w=w.double()),
                lambda: g(rows.double(), pos, 2)):
        with pytest.raises(TypeError):
            bad()
    out = torch.empty(6, 64, device=DEV)
    for bad in (lambda: f(out, pos, 2, out=out), lambda: g(rows[:6], pos, 2, y=rows[:6]),
                lambda: f(x[:, :60].contiguous(), pos, 2), lambda: h(x, x, pos, 2, drows=x)):
        with pytest.raises(gpu_lib.Nf4MoeError):
            bad()
