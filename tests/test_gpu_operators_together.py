"""The operators as they are used around the routed experts: a QLoRA step of one
block (norms, experts, gradients, adapter update) and a decode step (norms,
dense 4-bit projections, the expert layer)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import blocknorm, muon
from parity import half_spacing

pytestmark = pytest.mark.gpu
DEV = "cuda"
E, H, I, K, T, R = 8, 256, 128, 2, 48, 4
C = (3.4445, -4.7750, 2.0315)
U = 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def block(lib, seed=0):
    g = torch.Generator(DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    gu, dn = lib.quantize(n(E, 2 * I, H) * 0.05), lib.quantize(n(E, H, I) * 0.05)
    ad = dict(A_gu=n(E, R, H) * 0.05, B_gu=n(E, 2 * I, R) * 0.05, A_dn=n(E, R, I) * 0.05,
              B_dn=n(E, H, R) * 0.05)
    return dict(gu=gu, dn=dn, ad=ad, w_pre=1 + 0.1 * n(H), w_post=1 + 0.1 * n(H),
                router=n(H, E) * 0.1, x=n(T, H), target=n(T, H), gate=torch.sigmoid(n(T)))


class Step:
    """One block with its optimiser state; ``loss`` and ``step`` as a training loop
    has them (the router's product is torch's)."""

    def __init__(self, lib, b):
        self.lib, self.b = lib, b
        self.m = {k: torch.zeros_like(v) for k, v in b["ad"].items()}
        self.a16 = {k: v.half() for k, v in b["ad"].items()}

    def lora(self):
        return dict(gu_lora=(self.a16["A_gu"], self.a16["B_gu"], 2.0),
                    dn_lora=(self.a16["A_dn"], self.a16["B_dn"], 2.0))

    def forward(self):
        b, lib = self.b, self.lib
        _, h = lib.block_norm(b["x"], w_pre=b["w_pre"], h_dtype=torch.float16)
        logits = h.float() @ b["router"]
        y = lib.moe_forward(h, logits, K, *b["gu"], *b["dn"], y_dtype=torch.float32, **self.lora())
        out, _ = lib.block_norm(b["x"], y=y, w_post=b["w_post"], gate=b["gate"], alpha=0.5)
        return h, logits, y, out

    def gradients(self):
        b, lib = self.b, self.lib
        h, logits, y, out = self.forward()
        d = (out - b["target"]) / T
        post = lib.block_norm_backward(None, d, out, y=y, w_post=b["w_post"], gate=b["gate"],
                                       alpha=0.5)
        # dy is sent through the experts at a scale that fp16 holds well
        dh, grads = lib.moe_backward(h, logits, (post["dy"] * 1024).half(), K, *b["gu"], *b["dn"],
                                     dx_dtype=torch.float32, **self.lora())
        grads = {k[1:]: v / 1024 for k, v in grads.items()}
        pre = lib.block_norm_backward(dh / 1024, post["dresidual"], b["x"], w_pre=b["w_pre"])
        return out, post, pre, grads, dh

    def step(self, grads, lr):
        self.lib.lora_muon_step(
            [dict(grad=grads[k], momentum=self.m[k], w=self.b["ad"][k], w16=self.a16[k],
                  rank_major=k[0] == "A", scale=0.5) for k in sorted(grads)], lr=lr)


def test_qlora_step(gpu_lib):
    b = block(gpu_lib)
    s = Step(gpu_lib, b)
    out, post, pre, grads, dh = s.gradients()
    h, logits, y, _ = s.forward()
    # each operator on what the others gave it
    ref, size = blocknorm.post(host(b["x"]), host(y), host(b["w_post"]), host(b["gate"])[:, None],
                               0.5, 1.0, 1e-6)
    assert np.all(np.abs(host(out) - ref) <= 40 * U * size)
    ref = blocknorm.backward(host(dh / 1024), host(post["dresidual"]), host(b["x"]), None,
                             host(b["w_pre"]), None, np.ones(()), 1.0, 1.0, 1e-6)
    for k, (v, size) in ref.items():
        assert np.all(np.abs(host(pre[k]) - v) <= (200 + T) * U * size), k
    before = {k: v.clone() for k, v in b["ad"].items()}
    s.step(grads, 0.02)
    for k, g in grads.items():
        m = host(s.m[k])
        assert np.array_equal(m, host(g))
        o = muon.newton_schulz(host(g) + float(np.float32(0.95)) * m, 5, C, 1e-7)
        w = muon.muon_weight(host(before[k]), o, 0.02, 0.0, 0.5)
        tol = 0.02 * 0.5 * 485 * U + 2 * U * np.abs(w) + half_spacing(w, "f32")
        assert np.all(np.abs(host(b["ad"][k]) - w) <= tol), k
        assert torch.equal(s.a16[k], b["ad"][k].half())


def test_qlora_step_gradient_is_the_loss_slope(gpu_lib):
    """The whole chain's gradient against differences of its loss."""
    b = block(gpu_lib, 1)
    s = Step(gpu_lib, b)
    loss = lambda: float(((s.forward()[3] - b["target"]).double() ** 2).sum() / (2 * T))  # noqa: E731
    _, post, pre, grads, _ = s.gradients()
    for name, t, g in (("w_post", b["w_post"], post["dw_post"]), ("gate", b["gate"], post["dgate"])):
        kept, d = t.clone(), g / g.norm() * 0.05 * t.norm()
        t.copy_(kept + d)
        up = loss()
        t.copy_(kept - d)
        down = loss()
        t.copy_(kept)
        want = 2 * float((g.double() * d.double()).sum())
        # the output is quadratic in each: only rounding remains (fp32 rows)
        assert abs((up - down) - want) <= 1e-3 * abs(want), (name, up - down, want)
    for k, g in grads.items():
        kept, d = s.a16[k].clone(), g / g.norm() * 0.05 * s.a16[k].float().norm()
        s.a16[k].copy_(kept.float() + d)
        plus, up = s.a16[k].double(), loss()
        s.a16[k].copy_(kept.float() - d)
        minus, down = s.a16[k].double(), loss()
        s.a16[k].copy_(kept)
        want = float((g.double() * (plus - minus)).sum())
        # fp16 operands of the experts (2^-11 each) and a third derivative of a 5 % step
        assert abs((up - down) - want) <= 0.03 * abs(want), (k, up - down, want)


def test_training_loop_runs_in_a_graph(gpu_lib):
    """The update and the norms of a step captured and replayed as eager calls."""
    runs = []
    for graph in (False, True):
        b = block(gpu_lib, 2)
        s = Step(gpu_lib, b)
        grads = s.gradients()[3]
        if graph:
            keep = {k: (s.b["ad"][k].clone(), s.m[k].clone(), s.a16[k].clone()) for k in grads}
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                s.step(grads, 0.02)
            torch.cuda.current_stream().wait_stream(side)
            for k, (w, m, a) in keep.items():
                s.b["ad"][k].copy_(w)
                s.m[k].copy_(m)
                s.a16[k].copy_(a)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                s.step(grads, 0.02)
        for _ in range(3):
            new = s.gradients()[3]
            for k in grads:
                grads[k].copy_(new[k])
            if graph:
                g.replay()
                torch.cuda.synchronize()
            else:
                s.step(grads, 0.02)
        runs.append({k: s.b["ad"][k].clone() for k in grads})
    for k in runs[0]:
        assert torch.equal(runs[0][k], runs[1][k]), k


def test_decode_step(gpu_lib):
    """One token: norm, a dense 4-bit projection added to the stream, norm, experts, norm, head."""
    b = block(gpu_lib, 3)
    g = torch.Generator(DEV).manual_seed(9)
    wo, so = gpu_lib.quantize(torch.randn(1, H, H, generator=g, device=DEV) * 0.05)
    wh, sh = gpu_lib.quantize(torch.randn(1, 1000, H, generator=g, device=DEV) * 0.05)
    x = b["x"][:1].bfloat16()
    _, h = gpu_lib.block_norm(x, w_pre=b["w_pre"])
    a = gpu_lib.nbit_matvec(h, wo[0], so[0])
    r, h = gpu_lib.block_norm(x, y=a, w_pre=b["w_pre"])
    y = gpu_lib.moe_forward(h, h.float() @ b["router"], K, *b["gu"], *b["dn"])
    r2, h2 = gpu_lib.block_norm(r, y=y, w_pre=b["w_pre"], w_post=b["w_post"])
    logits = gpu_lib.nbit_matvec(h2, wh[0], sh[0], out_dtype=torch.float32)
    ref, size = blocknorm.post(host(x), host(a), None, np.ones(()), 1.0, 1.0, 1e-6)
    assert np.all(np.abs(host(r) - ref) <= 4 * U * size + half_spacing(ref, "bf16"))
    ref, size = blocknorm.post(host(r), host(y), host(b["w_post"]), np.ones(()), 1.0, 1.0, 1e-6)
    assert np.all(np.abs(host(r2) - ref) <= 40 * U * size + half_spacing(ref, "bf16"))
    ref = blocknorm.pre(host(r2), host(b["w_pre"]), 1e-6)
    assert np.all(np.abs(host(h2) - ref) <= 40 * U * np.abs(ref) + half_spacing(ref, "bf16"))
    ref, mag = oracle.matvec(host(h2), wh[0].cpu().numpy(), sh[0].cpu().numpy(), "nf4", 64)
    assert np.all(np.abs(host(logits) - ref) <= (H / 32 + 64) * 2 * U * mag)


def test_two_streams_at_once(gpu_lib):
    """The same calls running on two streams do not disturb each other."""
    g = torch.Generator(DEV).manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    wo, so = gpu_lib.quantize(n(1, 4096, 2048) * 0.02)
    res, y, w = n(700, 1024), n(700, 1024), n(1024)
    dh, u, x = n(700, 1024), n(40, 16, 1500), n(5, 2048).half()

    def work():
        r, h = gpu_lib.block_norm(res, y=y, w_pre=w, w_post=w)
        d = gpu_lib.block_norm_backward(dh, None, r, y=y, w_pre=w, w_post=w)
        return [r, h, gpu_lib.nbit_matvec(x, wo[0], so[0]), gpu_lib.lora_orthogonalize(u),
                *(d[k] for k in sorted(d))]

    want = work()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(work())
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
