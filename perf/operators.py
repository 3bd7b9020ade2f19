"""Timed cases of the operators around the routed experts, with their plain forms.

Three families:

- ``matvec``: products of 1 to 64 activation rows with one 4-bit matrix that
  has group scales (nf4, fp4, int4 with zero points, MXFP4);
- ``norm_fwd`` / ``norm_bwd``: the RMS norms after and before a block, fused
  with the block's gate and residual scale, and their gradients;
- ``orth`` / ``muon``: per-expert adapter factors orthogonalised by
  Newton-Schulz products, alone and as the whole optimiser step.

``own = False`` computes every pass with elementary torch operations;
``own = True`` calls the library.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}

# Newton-Schulz coefficients of the quintic iteration, and its step count
NS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7

NF4 = (-1.0, -0.6961928010, -0.5250729322, -0.3949174285, -0.2844413221, -0.1847734004,
       -0.0910499766, 0.0, 0.0795803145, 0.1609301418, 0.2461122572, 0.3379151225,
       0.4407097399, 0.5626168847, 0.7229566574, 1.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one token through a square projection of the H = 2048 models
        dict(name="matvec_nf4_1tok", op="matvec", T=1, N=2048, K=2048, q="nf4", group=64,
             x="bf16", out="bf16", bias=False),
        # one token through a wide dense projection stored as int4 with zero points
        dict(name="matvec_int4_1tok_wide", op="matvec", T=1, N=28672, K=4096, q="int4", group=128,
             x="f16", out="f16", bias=False),
        # sixteen sequences decoding at once on released MXFP4 bytes, with a bias
        dict(name="matvec_mxfp4_16tok", op="matvec", T=16, N=11520, K=2880, q="mxfp4", group=32,
             x="bf16", out="bf16", bias=True),
        # four drafted tokens through a 4-bit output head, logits in fp32
        dict(name="matvec_nf4_head_4tok", op="matvec", T=4, N=151936, K=2048, q="nf4", group=64,
             x="bf16", out="f32", bias=False),
        # a ragged batch of more rows than one matrix-unit tile, odd output count
        dict(name="matvec_fp4_37tok_odd", op="matvec", T=37, N=5003, K=1088, q="fp4", group=64,
             x="f16", out="f16", bias=False),
        # decode: the residual of one token updated and normalised between two blocks
        dict(name="norm_fwd_1tok", op="norm_fwd", T=1, H=2048, res="bf16", y="bf16", w="bf16",
             post=True, gate="none", dres=True),
        # prefill: both norms around an expert block, each token's gate on its output
        dict(name="norm_fwd_4096", op="norm_fwd", T=4096, H=2048, res="bf16", y="bf16", w="bf16",
             post=True, gate="token", dres=True),
        # training: the gradients of the same
        dict(name="norm_bwd_4096", op="norm_bwd", T=4096, H=2048, res="bf16", y="bf16", w="bf16",
             post=True, gate="token", dres=True),
        # training with an fp32 residual stream, a gate per channel, ragged sizes
        dict(name="norm_bwd_f32_odd", op="norm_bwd", T=1531, H=2888, res="f32", y="f16", w="f32",
             post=True, gate="channel", dres=True),
        # the update of one small adapter, orthogonalised by itself
        dict(name="orth_8x8x1000", op="orth", E=8, r=8, n=1000, major="rank", u="f32", out="f32"),
        # the optimiser step of all four adapter factors of an OLMoE layer (E64 H2048 I1024, r 8)
        dict(name="muon_olmoe_r8", op="muon", E=64, r=8, H=2048, I=1024, w="f32"),
        # the same for a Qwen3-30B-A3B layer (E128 H2048 I768) at rank 16, bf16 adapters
        dict(name="muon_qwen3_r16", op="muon", E=128, r=16, H=2048, I=768, w="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "norm_fwd", "norm_bwd", "orth", "muon"])
    if op == "matvec":
        q = rng.choice(["nf4", "fp4", "int4", "mxfp4"])
        group = {"nf4": 64, "fp4": 64, "mxfp4": 32}.get(q) or rng.choice([32, 64, 128])
        K = max(1, _log(rng, 256, 16384) // group) * group
        T = _log(rng, 1, 64)
        # no larger than the output head in bytes, nor more than its products
        N = _log(rng, 16, min(150000, max(32, 300000000 // K), max(32, 1200000000 // (K * T))))
        return dict(op=op, T=T, N=N, K=K, q=q, group=group, x=rng.choice(["bf16", "f16"]),
                    out=rng.choice(["bf16", "f16", "f32"]), bias=rng.random() < 0.3)
    if op in ("norm_fwd", "norm_bwd"):
        H = max(1, _log(rng, 128, 16384) // 8) * 8
        T = _log(rng, 1, max(2, 6000000 // H))
        return dict(op=op, T=T, H=H, res=rng.choice(["bf16", "f16", "f32"]),
                    y=rng.choice(["bf16", "f16", "f32"]), w=rng.choice(["bf16", "f32"]),
                    post=rng.random() < 0.6, gate=rng.choice(["none", "token", "channel"]),
                    dres=rng.random() < 0.7)
    r = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16, 16])
    E = _log(rng, 1, 128)
    if op == "orth":
        return dict(op=op, E=E, r=r, n=_log(rng, 16, 8192), major=rng.choice(["rank", "long"]),
                    u=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16", "f16"]))
    H = max(1, _log(rng, 64, 4096) // 64) * 64
    I = max(1, _log(rng, 64, 2048) // 64) * 64
    E = max(1, min(E, 9000000 // (r * (2 * H + 3 * I))))
    return dict(op=op, E=E, r=r, H=H, I=I, w=rng.choice(["f32", "bf16", "f16"]))


# ---- inputs ---------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, T, width, dtype):
    """Unit-variance rows with a few channels twenty times as large."""
    x = _randn(g, T, width)
    ch = torch.randint(0, width, (max(1, width // 256),), generator=g, device=DEV)
    x[:, ch] *= 20.0
    return x.to(dtype)


def _pack(codes):
    """Codes [N, K] -> bytes [N, K/2], the even element in the high nibble."""
    c = codes.to(torch.uint8)
    return (c[:, 0::2] << 4) | c[:, 1::2]


def _weights(g, N, K, q, group):
    """A quantised N(0, 0.02) matrix: (codes u8 [N, K/2], scales, zeros)."""
    w = _randn(g, N, K).view(N, K // group, group) * 0.02
    if q in ("nf4", "fp4"):
        s = w.abs().amax(2)
        xn = w / s[:, :, None]
        if q == "nf4":
            lv = torch.tensor(NF4, device=DEV)
            codes = torch.bucketize(xn, (lv[1:] + lv[:-1]) / 2, out_int32=True)
        else:
            lv = torch.tensor(E2M1[:8], device=DEV) / 6.0
            codes = torch.bucketize(xn.abs(), (lv[1:] + lv[:-1]) / 2, out_int32=True)
            codes = codes + 8 * (xn < 0)
        return _pack(codes.view(N, K)), s.contiguous(), None
    if q == "mxfp4":
        e = torch.floor(torch.log2(w.abs().amax(2))) - 2
        xn = w / torch.exp2(e)[:, :, None]
        lv = torch.tensor(E2M1[:8], device=DEV)
        codes = torch.bucketize(xn.abs(), (lv[1:] + lv[:-1]) / 2, out_int32=True) + 8 * (xn < 0)
        b = codes.view(N, K).to(torch.uint8)
        return b[:, 0::2] | (b[:, 1::2] << 4), (e + 127).to(torch.uint8).contiguous(), None
    lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
    s = ((hi - lo) / 15).half()
    z = torch.round(-lo / s.float()).clamp(0, 15)
    codes = (torch.round(w / s.float()[:, :, None]) + z[:, :, None]).clamp(0, 15)
    return _pack(codes.view(N, K)), s.contiguous(), z.to(torch.uint8).contiguous()


def _spectrum(g, E, r, n, major):
    """Gradient-like factors: singular values spread over two decades, each
    expert of its own size, and every sixteenth expert without rows (zeros)."""
    u = _randn(g, E, r, n)
    mix = _randn(g, E, r, r) / math.sqrt(r)
    fall = torch.logspace(0, -2, r, device=DEV) if r > 1 else torch.ones(1, device=DEV)
    u = torch.matmul(mix, u * fall[None, :, None])
    u = u * torch.exp2(4 * _randn(g, E, 1, 1)) * 1e-3
    u[7::16] = 0
    return (u if major == "rank" else u.transpose(1, 2)).contiguous()


def _factors(case):
    """(name, long axis, layout) of the four adapter factors of a layer."""
    return [("A_gu", case["H"], "rank"), ("B_gu", 2 * case["I"], "long"),
            ("A_dn", case["I"], "rank"), ("B_dn", case["H"], "long")]


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "matvec":
        T, N, K = case["T"], case["N"], case["K"]
        st["xv"] = _activations(g, T, K, TYPES[case["x"]])
        st["codes"], st["scales"], st["zeros"] = _weights(g, N, K, case["q"], case["group"])
        st["b"] = _randn(g, N) * 0.1 if case["bias"] else None
    elif op in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        st["residual"] = (3 * _activations(g, T, H, torch.float32)).to(TYPES[case["res"]])
        st["yv"] = (0.5 * _randn(g, T, H)).to(TYPES[case["y"]])
        wt = TYPES[case["w"]]
        st["w_pre"] = (1 + 0.1 * _randn(g, H)).to(wt)
        st["w_post"] = (1 + 0.1 * _randn(g, H)).to(wt) if case["post"] else None
        n = {"token": T, "channel": H}.get(case["gate"])
        st["gatev"] = torch.sigmoid(_randn(g, n)) if n else None
        if op == "norm_bwd":
            # r as a forward pass stores it
            st["r"] = (0.7 * st["residual"].float() + 0.5 * _randn(g, T, H)).to(TYPES[case["res"]])
            st["dh"] = (0.01 * _randn(g, T, H)).to(torch.bfloat16)
            st["drv"] = (0.01 * _randn(g, T, H)).to(TYPES[case["res"]]) if case["dres"] else None
            del st["residual"]
    elif op == "orth":
        st["uv"] = _spectrum(g, case["E"], case["r"], case["n"], case["major"]).to(
            TYPES[case["u"]])
    else:
        E, r = case["E"], case["r"]
        st["t"] = []
        for name, n, major in _factors(case):
            d = dict(name=name, n=n, major=major)
            d["g"] = _spectrum(g, E, r, n, major)
            d["m"] = _spectrum(g, E, r, n, major) * 3
            d["w"] = (0.01 * _randn(g, *d["g"].shape)).to(TYPES[case["w"]])
            d["m_out"], d["w_out"] = torch.empty_like(d["m"]), torch.empty_like(d["w"])
            # fp32 master factors come with the 16-bit copy that the layer reads
            d["w16"] = torch.empty_like(d["w"], dtype=torch.bfloat16) if case["w"] == "f32" \
                else None
            st["t"].append(d)
    return st


# norm scales and the optimiser's numbers
EPS, ALPHA, BETA = 1e-6, 0.5, 0.7
LR, MU, WD, UPDATE = 0.02, 0.95, 0.1, 0.2


# ---- the passes -----------------------------------------------------------

def run(st):
    return (_own if own else _plain)[st["op"]](st)


def _plain_weight(st):
    """The matrix as fp32 [N, K]."""
    c, q = st["codes"], st["q"]
    hi, lo = c >> 4, c & 15
    pair = (lo, hi) if q == "mxfp4" else (hi, lo)
    idx = torch.stack(pair, 2).view(c.shape[0], -1).int()
    if q == "nf4":
        v = torch.tensor(NF4, device=DEV)[idx]
        s = st["scales"]
    elif q == "int4":
        v, s = idx.float(), st["scales"].float()
    else:
        v = torch.tensor(E2M1, device=DEV)[idx]
        s = st["scales"] / 6.0 if q == "fp4" else torch.exp2(st["scales"].float() - 127)
    v = v.view(c.shape[0], -1, st["group"])
    if q == "int4":
        v = v - st["zeros"].float()[:, :, None]
    return (v * s[:, :, None]).view(c.shape[0], -1)


def _plain_matvec(st):
    y = torch.matmul(st["xv"].float(), _plain_weight(st).t())
    if st["b"] is not None:
        y = y + st["b"]
    return y.to(TYPES[st["out"]])


def _plain_gate(st):
    if st["gatev"] is None:
        return 1.0
    return st["gatev"][:, None] if st["gate"] == "token" else st["gatev"][None, :]


def _plain_norm_fwd(st):
    y = st["yv"].float()
    if st["post"]:
        y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * st["w_post"].float()
    r = BETA * st["residual"].float() + ALPHA * _plain_gate(st) * y
    r = r.to(TYPES[st["res"]])
    x = r.float()
    h = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * st["w_pre"].float()
    return r, h.to(torch.bfloat16)


def _plain_rms_grad(gy, x, w):
    """Gradients of x * rstd * w: (dx, dw)."""
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    gw = gy * w
    dx = rstd * gw - x * rstd ** 3 * (gw * x).mean(1, keepdim=True)
    return dx, (gy * x * rstd).sum(0)


def _plain_norm_bwd(st):
    dr, dw_pre = _plain_rms_grad(st["dh"].float(), st["r"].float(), st["w_pre"].float())
    if st["drv"] is not None:
        dr = dr + st["drv"].float()
    y = st["yv"].float()
    z = y
    if st["post"]:
        z = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * st["w_post"].float()
    out = dict(dresidual=(BETA * dr).to(TYPES[st["res"]]), dw_pre=dw_pre)
    if st["gatev"] is not None:
        out["dgate"] = ALPHA * (dr * z).sum(1 if st["gate"] == "token" else 0)
    dy = ALPHA * _plain_gate(st) * dr
    if st["post"]:
        dy, out["dw_post"] = _plain_rms_grad(dy, y, st["w_post"].float())
    out["dy"] = dy.to(TYPES[st["y"]])
    return out


def _plain_ns(u, major):
    """Newton-Schulz on [E, r, n] (or [E, n, r]); the smallest singular
    values grow 485-fold over the steps and errors with them, so in 64 bits."""
    x = (u if major == "rank" else u.transpose(1, 2)).double().contiguous()
    x = x / ((x * x).sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    a, b, c = NS
    for _ in range(NS_STEPS):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return x if major == "rank" else x.transpose(1, 2).contiguous()


def _plain_orth(st):
    return _plain_ns(st["uv"], st["major"]).to(TYPES[st["out"]])


def _plain_muon(st):
    out = {}
    for d in st["t"]:
        m = MU * d["m"] + d["g"]
        o = _plain_ns(d["g"] + MU * m, d["major"])
        w = (1 - LR * WD) * d["w"].double() - LR * UPDATE * o
        out[d["name"]] = [m, w.to(TYPES[st["w"]])]
        if d["w16"] is not None:
            out[d["name"]].append(w.float().to(torch.bfloat16))
    return out


_plain = dict(matvec=_plain_matvec, norm_fwd=_plain_norm_fwd, norm_bwd=_plain_norm_bwd,
              orth=_plain_orth, muon=_plain_muon)


def _lib():
    from grouped_nf4_gemm_quantize_amd import binding

    return binding


def _own_matvec(st):
    return _lib().nbit_matvec(st["xv"], st["codes"], st["scales"], quant_type=st["q"],
                              group=st["group"], zeros=st["zeros"], bias=st["b"],
                              out_dtype=TYPES[st["out"]])


def _own_norm_fwd(st):
    return _lib().block_norm(st["residual"], y=st["yv"], w_pre=st["w_pre"], w_post=st["w_post"],
                             gate=st["gatev"], gate_axis=st["gate"], alpha=ALPHA, beta=BETA,
                             eps=EPS, h_dtype=torch.bfloat16)


def _own_norm_bwd(st):
    return _lib().block_norm_backward(st["dh"], st["drv"], st["r"], y=st["yv"],
                                      w_pre=st["w_pre"], w_post=st["w_post"], gate=st["gatev"],
                                      gate_axis=st["gate"], alpha=ALPHA, beta=BETA, eps=EPS)


def _own_orth(st):
    return _lib().lora_orthogonalize(st["uv"], rank_major=st["major"] == "rank", steps=NS_STEPS,
                                     coeffs=NS, eps=NS_EPS, out_dtype=TYPES[st["out"]])


def _own_muon(st):
    _lib().lora_muon_step(
        [dict(grad=d["g"], momentum=d["m"], w=d["w"], rank_major=d["major"] == "rank",
              scale=UPDATE, momentum_out=d["m_out"], w_out=d["w_out"], w16=d["w16"])
         for d in st["t"]],
        lr=LR, momentum=MU, nesterov=True, weight_decay=WD, steps=NS_STEPS, coeffs=NS,
        eps=NS_EPS)
    return {d["name"]: [x for x in (d["m_out"], d["w_out"], d["w16"]) if x is not None]
            for d in st["t"]}


_own = dict(matvec=_own_matvec, norm_fwd=_own_norm_fwd, norm_bwd=_own_norm_bwd,
            orth=_own_orth, muon=_own_muon)


# ---- what a pass cannot do without ----------------------------------------

def work(case):
    op = case["op"]
    if op == "matvec":
        T, N, K, G = case["T"], case["N"], case["K"], case["group"]
        per = {"nf4": 4, "fp4": 4, "mxfp4": 1, "int4": 3}[case["q"]]
        b = N * K // 2 + per * N * (K // G) + 2 * T * K + BYTES[case["out"]] * T * N
        return dict(bytes=b + (4 * N if case["bias"] else 0), flops=2 * T * N * K)
    if op in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        rb, yb, wb = BYTES[case["res"]], BYTES[case["y"]], BYTES[case["w"]]
        n = 4 * {"token": T, "channel": H}.get(case["gate"], 0)
        norms = 2 if case["post"] else 1
        if op == "norm_fwd":
            return dict(bytes=T * H * (2 * rb + yb + 2) + n + norms * H * wb,
                        flops=T * H * (3 + 5 * norms))
        b = T * H * (2 + 2 * rb + 2 * yb + (rb if case["dres"] else 0))
        return dict(bytes=b + 2 * n + norms * H * (wb + 4), flops=T * H * (5 + 11 * norms))
    E, r = case["E"], case["r"]
    if op == "orth":
        n = E * r * case["n"]
        return dict(bytes=n * (BYTES[case["u"]] + BYTES[case["out"]]), flops=4 * r * n)
    n = sum(E * r * f[1] for f in _factors(case))
    wb = BYTES[case["w"]]
    return dict(bytes=n * (12 + 2 * wb + (2 if case["w"] == "f32" else 0)), flops=n * (4 * r + 8))


# ---- the definitions in 64 bits -------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f8 = torch.float64
    if op == "matvec":
        T, N, K, G, q = case["T"], case["N"], case["K"], case["group"], case["q"]
        table = torch.tensor(NF4 if q == "nf4" else E2M1 if q != "int4" else range(16),
                             device=DEV, dtype=torch.float32 if q == "nf4" else f8).to(f8)
        if q == "fp4":
            table = table / 6
        x = st["xv"].to(f8)
        x0, x1 = x[:, 0::2].contiguous(), x[:, 1::2].contiguous()
        y = torch.zeros(T, N, dtype=f8, device=DEV)
        at = max(1, (1 << 26) // K)
        for n in range(0, N, at):  # some rows at a time: the matrix in 64 bits is large
            c = st["codes"][n:n + at]
            first, second = ((c & 15), (c >> 4)) if q == "mxfp4" else ((c >> 4), (c & 15))
            s = st["scales"][n:n + at].to(f8)
            if q == "mxfp4":
                s = torch.pow(torch.tensor(2.0, dtype=f8, device=DEV), s - 127)
            s = s.repeat_interleave(G // 2, 1)
            z = 0.0
            if q == "int4":
                z = st["zeros"][n:n + at].to(f8).repeat_interleave(G // 2, 1)
            for codes, xs in ((first, x0), (second, x1)):
                w = (table[codes.int()] - z) * s
                y[:, n:n + at] += torch.matmul(xs, w.t().contiguous())
        return y if st["b"] is None else y + st["b"].to(f8)
    if op == "norm_fwd":
        y, res = st["yv"].to(f8), st["residual"].to(f8)
        H = y.shape[1]
        if case["post"]:
            y = st["w_post"].to(f8) * y / torch.sqrt(y.square().sum(1, True) / H + EPS)
        gv = torch.ones(1, 1, dtype=f8, device=DEV) if st["gatev"] is None else \
            st["gatev"].to(f8).reshape((-1, 1) if case["gate"] == "token" else (1, -1))
        r = res * BETA + y * gv * ALPHA
        # h is defined on r as it is stored
        x = r.to(TYPES[case["res"]]).to(f8) if case["res"] != "f32" else r
        return r, st["w_pre"].to(f8) * x / torch.sqrt(x.square().sum(1, True) / H + EPS)
    if op == "norm_bwd":
        # by differentiating the definition
        leaf = lambda t: None if t is None else t.to(f8).requires_grad_()  # noqa: E731
        r, y, w1, w2, gv = (leaf(st[k]) for k in ("r", "yv", "w_pre", "w_post", "gatev"))
        H = r.shape[1]
        h = w1 * r / torch.sqrt(r.square().sum(1, True) / H + EPS)
        dr, dw1 = torch.autograd.grad(h, [r, w1], st["dh"].to(f8))
        if st["drv"] is not None:
            dr = dr + st["drv"].to(f8)
        z = y if w2 is None else w2 * y / torch.sqrt(y.square().sum(1, True) / H + EPS)
        s = z * ALPHA
        if gv is not None:
            s = s * (gv[:, None] if case["gate"] == "token" else gv)
        want = dict(dy=y, dw_post=w2, dgate=gv)
        want = {k: v for k, v in want.items() if v is not None}
        got = torch.autograd.grad(s, list(want.values()), dr)
        return dict(zip(want, got), dresidual=BETA * dr, dw_pre=dw1)

    def polar(u, major):
        # the iteration acts on the singular values alone: p(s) five times
        t = u.to(f8).cpu()
        t = t if major == "rank" else t.transpose(1, 2)
        t = t / (t.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
        U, S, V = torch.linalg.svd(t, full_matrices=False)
        for _ in range(NS_STEPS):
            S = S * (NS[0] + S * S * (NS[1] + NS[2] * S * S))
        t = torch.matmul(U * S[:, None, :], V)
        return (t if major == "rank" else t.transpose(1, 2)).contiguous().to(DEV)

    if op == "orth":
        return polar(st["uv"], case["major"])
    out = {}
    for d in st["t"]:
        m = d["g"].to(f8) + d["m"].to(f8) * MU
        w = d["w"].to(f8) - LR * (WD * d["w"].to(f8) + UPDATE * polar(m * MU + d["g"].to(f8),
                                                                      d["major"]))
        out[d["name"]] = [m, w] + ([w] if d["w16"] is not None else [])
    return out
