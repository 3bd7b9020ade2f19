"""Block norms and their gradients on the GPU against 64 bits.

Tolerances count roundings of 2^-24.  A mean over H of squares goes through at
most 16 sums in a thread, 6 in a wave and 16 over waves, and rstd halves its error:
h has |h| * 32 * 2^-24 plus half a step of its type.  r has three roundings of its
terms plus half a step, and z's 32.  Gradients add two such sums: 96 of the sum
of their terms' sizes.  Sums over T have T terms at most in order: (96 + T).
"""

import numpy as np
import pytest
import torch

from oracle import blocknorm
from parity import half_spacing

pytestmark = pytest.mark.gpu
DEV = "cuda"
TT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def make(T, H, res="bf16", y="bf16", w="f32", post=True, pre=True, gate="token", h="bf16",
         d_r=True, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * T + H)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = dict(residual=(3 * n(T, H)).to(TT[res]), y=n(T, H).to(TT[y]) if y else None,
             w_pre=n(H).to(TT[w]) if pre else None, w_post=n(H).to(TT[w]) if post else None,
             gate=None, dh=n(T, H).to(TT[h]) if pre else None,
             d_r=n(T, H).to(TT[res]) if d_r else None)
    if gate != "none":
        c["gate"] = n(T if gate == "token" else H)
    return {k: None if v is None else v.to(DEV) for k, v in c.items()}


def wide(gate, axis):
    if gate is None:
        return np.ones(())
    return host(gate)[:, None] if axis == "token" else host(gate)[None, :]


def near(got, ref, size, count, out):
    tol = count * U * size + half_spacing(ref, out)
    d = np.abs(host(got) - ref)
    assert not (d > tol).any(), (np.argwhere(d > tol)[:4], (d / np.maximum(tol, 1e-300)).max())


def both(lib, c, T, H, res="bf16", y="bf16", h="bf16", gate="token", alpha=0.5, beta=0.7,
         eps=1e-6, off=0.0):
    """Forward and backward of one case against the oracle."""
    kw = dict(y=c["y"], w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"], gate_axis=gate,
              alpha=alpha, beta=beta, eps=eps, w_offset=off)
    r, hh = lib.block_norm(c["residual"], h_dtype=TT[h], **kw)
    plus = lambda w: None if w is None else host(w) + off  # noqa: E731
    gv = wide(c["gate"], gate)
    if c["y"] is None:
        assert r is c["residual"]
    else:
        ref, size = blocknorm.post(host(c["residual"]), host(c["y"]), plus(c["w_post"]), gv, alpha,
                                   beta, eps)
        near(r, ref, size, 36, res)
    if c["w_pre"] is None:
        assert hh is None
    else:
        ref = blocknorm.pre(host(r), plus(c["w_pre"]), eps)
        near(hh, ref, np.abs(ref), 36, h)
    g = lib.block_norm_backward(c["dh"], c["d_r"], r, **kw)
    ref = blocknorm.backward(None if c["dh"] is None else host(c["dh"]),
                             None if c["d_r"] is None else host(c["d_r"]), host(r),
                             None if c["y"] is None else host(c["y"]), plus(c["w_pre"]),
                             plus(c["w_post"]), gv, alpha, beta, eps)
    assert set(g) == set(ref)
    for k, (v, size) in ref.items():
        out = {"dresidual": res, "dy": y}.get(k, "f32")
        count = 96 if out != "f32" or k in ("dresidual", "dy") else 96 + T + 64
        if k == "dgate" and gate == "token":
            count = 96 + 64
        near(g[k], v.reshape(g[k].shape), size.reshape(g[k].shape), count, out)
    return r, hh, g


@pytest.mark.parametrize("H", [8, 64, 72, 512, 520, 2048, 2888, 4104, 8192, 8200, 16384])
@pytest.mark.parametrize("T", [1, 3, 130])
def test_sizes(gpu_lib, T, H):
    both(gpu_lib, make(T, H), T, H)


@pytest.mark.parametrize("H", [24, 512, 1000, 2048, 2888, 5120, 8200, 16384])
@pytest.mark.parametrize("T", [2, 275])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_channel_gate_sizes(gpu_lib, T, H, t):
    """Every split of a row over waves, several rows a workgroup, with the sums over T."""
    both(gpu_lib, make(T, H, res=t, y=t, h=t, gate="channel"), T, H, res=t, y=t, h=t, gate="channel")


def test_many_long_rows(gpu_lib):
    """Three rows of 16 columns a lane for most workgroups."""
    both(gpu_lib, make(530, 8208), 530, 8208)


@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre,d_r", [(True, True), (True, False), (False, True)])
def test_parts(gpu_lib, gate, post, pre, d_r):
    T, H = 67, 768
    both(gpu_lib, make(T, H, post=post, pre=pre, gate=gate, d_r=d_r), T, H, gate=gate)


@pytest.mark.parametrize("d_r", [True, False])
def test_norm_alone(gpu_lib, d_r):
    T, H = 33, 2048
    both(gpu_lib, make(T, H, y=None, post=False, gate="none", d_r=d_r), T, H, gate="none", beta=1.0)


@pytest.mark.parametrize("res,y,h,w", [("f32", "bf16", "bf16", "bf16"), ("f16", "f16", "f16", "f16"),
                                       ("bf16", "f32", "f32", "bf16"), ("f32", "f32", "f32", "f32"),
                                       ("f32", "f16", "f16", "f32"), ("f16", "bf16", "f32", "bf16")])
def test_types(gpu_lib, res, y, h, w):
    T, H = 21, 1032
    both(gpu_lib, make(T, H, res=res, y=y, h=h, w=w), T, H, res=res, y=y, h=h)


def test_many_rows_and_scalars(gpu_lib):
    T, H = 2500, 264
    both(gpu_lib, make(T, H, gate="channel"), T, H, gate="channel", alpha=-1.5, beta=1.25, eps=1e-3,
         off=1.0)


def test_zero_rows_and_eps_zero(gpu_lib):
    """A row of zeros has rstd = eps^-1/2 and stays finite; eps = 0 is allowed."""
    T, H = 5, 256
    c = make(T, H)
    c["y"][2] = 0
    c["residual"][2] = 0
    r, h, g = both(gpu_lib, c, T, H, eps=1e-6)
    assert torch.count_nonzero(r[2]) == 0 and torch.count_nonzero(h[2]) == 0
    assert all(torch.isfinite(v).all() for v in g.values())
    both(gpu_lib, make(T, H), T, H, eps=0.0)


def test_rows_of_small_values_without_eps(gpu_lib):
    """rstd of some 1e14: its third power is beyond fp32, the gradients are not."""
    T, H = 9, 520
    c = make(T, H, res="f32", y="f32", h="f32")
    c["residual"] *= 1e-14
    c["y"] *= 1e-14
    _, _, g = both(gpu_lib, c, T, H, res="f32", y="f32", h="f32", alpha=1e-14, eps=0.0)
    assert all(torch.isfinite(v).all() for v in g.values())


def test_non_finite_rows_stay_alone(gpu_lib):
    T, H = 9, 512
    c = make(T, H)
    kw = dict(w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"])
    r0, h0 = gpu_lib.block_norm(c["residual"], y=c["y"], **kw)
    y = c["y"].clone()
    y[4, 3] = float("nan")
    y[6, 5] = float("inf")
    r, h = gpu_lib.block_norm(c["residual"], y=y, **kw)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(r[keep], r0[keep]) and torch.equal(h[keep], h0[keep])
    assert torch.isnan(h[4]).all() and torch.isnan(h[6]).any()


def test_in_place_and_fused_is_separate(gpu_lib):
    T, H = 40, 1024
    c = make(T, H)
    kw = dict(w_post=c["w_post"], gate=c["gate"], alpha=0.5)
    r, h = gpu_lib.block_norm(c["residual"], y=c["y"], w_pre=c["w_pre"], **kw)
    r1, none = gpu_lib.block_norm(c["residual"], y=c["y"], **kw)
    assert none is None and torch.equal(r1, r)
    assert torch.equal(gpu_lib.block_norm(r1, w_pre=c["w_pre"])[1], h)
    res, y = c["residual"].clone(), c["y"].clone()
    r2, h2 = gpu_lib.block_norm(res, y=y, w_pre=c["w_pre"], r_out=res, h=y, **kw)
    assert r2 is res and h2 is y and torch.equal(res, r) and torch.equal(y, h)


def test_backward_repeats_and_graph_replays(gpu_lib):
    T, H = 700, 640
    c = make(T, H, gate="channel")
    kw = dict(y=c["y"], w_pre=c["w_pre"], w_post=c["w_post"], gate=c["gate"], gate_axis="channel")
    r, _ = gpu_lib.block_norm(c["residual"], **kw)
    want = gpu_lib.block_norm_backward(c["dh"], c["d_r"], r, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gpu_lib.block_norm_backward(c["dh"], c["d_r"], r, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = gpu_lib.block_norm_backward(c["dh"], c["d_r"], r, **kw)
    for i in range(3):
        c["dh"].copy_(torch.randn(T, H, device=DEV, generator=torch.Generator(DEV).manual_seed(i)))
        for v in got.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = gpu_lib.block_norm_backward(c["dh"], c["d_r"], r, **kw)
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_gradient_by_differences(gpu_lib):
    """fp32 throughout: the loss along a direction against the gradient's."""
    T, H = 6, 64
    c = make(T, H, res="f32", y="f32", h="f32", gate="token")
    p = {k: c[k] for k in ("residual", "y", "w_pre", "w_post", "gate")}
    f = lambda q: gpu_lib.block_norm(q["residual"], y=q["y"], w_pre=q["w_pre"],  # noqa: E731
                                     w_post=q["w_post"], gate=q["gate"], alpha=0.5, eps=1e-2)

    def loss(q):
        r, h = f(q)
        return float((r.double() * c["d_r"].double()).sum() + (h.double() * c["dh"].double()).sum())

    r, _ = f(p)
    g = gpu_lib.block_norm_backward(c["dh"], c["d_r"], r, y=p["y"], w_pre=p["w_pre"],
                                    w_post=p["w_post"], gate=p["gate"], alpha=0.5, eps=1e-2)
    names = dict(residual="dresidual", y="dy", w_pre="dw_pre", w_post="dw_post", gate="dgate")
    for i, (k, name) in enumerate(names.items()):
        d = torch.randn(p[k].shape, device=DEV, generator=torch.Generator(DEV).manual_seed(i))
        step = 1.0 / 64
        num = (loss(dict(p, **{k: p[k] + step * d})) - loss(dict(p, **{k: p[k] - step * d}))) / (
            2 * step)
        want = float((g[name].double() * d.double()).sum())
        # a third derivative times step^2 / 6 and 2 T H roundings of 2^-24 over the step
        size = float((g[name].double() * d.double()).abs().sum())
        assert abs(num - want) < 2e-3 * size, (k, num, want, size)


def test_binding_refuses_on_the_gpu(gpu_lib):
    c = make(4, 64)
    for bad in (dict(y=c["y"][:3]), dict(w_pre=c["w_pre"][:32]), dict(gate=c["gate"][:2]),
                dict(y=c["y"].cpu()), dict(r_out=torch.empty(4, 72, device=DEV)),
                dict(gate=c["gate"], gate_axis="channel")):
        with pytest.raises(ValueError):
            gpu_lib.block_norm(c["residual"], **dict(dict(y=c["y"], w_pre=c["w_pre"]), **bad))
    with pytest.raises(TypeError):
        gpu_lib.block_norm(c["residual"], y=c["y"], w_pre=c["w_pre"], w_post=c["w_post"].half())
    with pytest.raises(gpu_lib.Nf4MoeError):
        gpu_lib.block_norm(c["residual"])
    with pytest.raises(gpu_lib.Nf4MoeError):
        gpu_lib.block_norm_backward(c["dh"], None, c["residual"])
