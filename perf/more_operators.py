"""Timed cases of microscaled 4-bit products and of the expert rows' way, with their plain forms.

Two families:

- ``quant``: MXFP4 blocks made of a matrix or a stack (along its rows, or along
  its columns for the transposed product) and read back; ``product``: activation
  rows quantised and multiplied with an MXFP4 stack, by expert, 4 bits by 4 bits;
- ``dispatch``, ``combine``, ``combine_bwd``: token rows into expert order, the
  experts' rows back into tokens with the routing weights, and the gradients of
  that for the rows, the weights and the router's logits.

``own = False`` computes every pass with elementary torch operations;
``own = True`` calls the library.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # decode: one token's activations through the format and back
        dict(name="quant_1tok", op="quant", E=1, R=1, K=2048, x="bf16", out="bf16", cols=False),
        # load time: expert matrices blocked along their outputs, for the product's input gradient
        dict(name="quant_stack_cols", op="quant", E=16, R=2048, K=2048, x="bf16", out="bf16",
             cols=True),
        # decode: one token through the gate and up projections of its 8 experts (E64 H2048 I1024)
        dict(name="product_1tok", op="product", T=1, E=64, k=8, K=2048, N=2048, x="bf16",
             out="f16", swiglu=True, spread=0.0),
        # prefill: the same layer with 4096 tokens
        dict(name="product_4096tok", op="product", T=4096, E=64, k=8, K=2048, N=2048, x="bf16",
             out="f16", swiglu=True, spread=0.0),
        # a ragged prompt on 32 experts of 2880 columns, a few of them crowded, fp32 out
        dict(name="product_333tok_odd", op="product", T=333, E=32, k=4, K=2880, N=5760, x="f16",
             out="f32", swiglu=False, spread=2.0),
        # a large dense projection: one matrix, every row its own
        dict(name="product_dense_8192", op="product", T=8192, E=1, k=1, K=8192, N=8192, x="bf16",
             out="bf16", swiglu=False, spread=0.0),
        # decode: sixteen tokens into the order of their experts
        dict(name="dispatch_16tok", op="dispatch", T=16, E=128, k=8, H=2048, x="bf16", out="f16",
             weights=False, drop=0.0),
        # prefill or training: 4096 tokens
        dict(name="dispatch_4096tok", op="dispatch", T=4096, E=64, k=8, H=2048, x="bf16",
             out="f16", weights=False, drop=0.0),
        # the experts' rows back into the tokens, weighted
        dict(name="combine_4096tok", op="combine", T=4096, E=64, k=8, H=2048, x="f16", out="bf16",
             weights=True, drop=0.0),
        # the gradient of a dispatch that dropped what was over the experts' capacity, ragged
        dict(name="combine_777tok_odd", op="combine", T=777, E=32, k=4, H=2888, x="f32", out="f32",
             weights=False, drop=0.1),
        # training: gradients for the experts' rows, the routing weights and the logits
        dict(name="combine_bwd_4096tok", op="combine_bwd", T=4096, E=64, k=8, H=2048, x="bf16",
             rows="f16", out="f16", renorm=True, drop=0.0),
        # the same for a ragged batch on many experts, weights of the whole softmax
        dict(name="combine_bwd_777tok_odd", op="combine_bwd", T=777, E=128, k=6, H=1448, x="f32",
             rows="bf16", out="bf16", renorm=False, drop=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "dispatch", "combine", "combine_bwd"])
    any_type = lambda: rng.choice(["f32", "bf16", "f16"])  # noqa: E731
    if op == "quant":
        cols = rng.random() < 0.5
        E = _log(rng, 1, 64)
        K = _log(rng, 1, 256) * BLOCK
        R = _log(rng, 1, max(2, min(65536, 67000000 // (E * K))))
        if cols:  # blocks run along R then, K may be anything
            R, K = max(1, R // BLOCK) * BLOCK, max(1, K - rng.choice([0, 0, 8, 31]))
        return dict(op=op, E=E, R=R, K=K, x=any_type(), out=any_type(), cols=cols)
    if op == "product":
        E = _log(rng, 1, 128)
        k = rng.randint(1, min(E, 8))
        K = _log(rng, 4, 256) * BLOCK
        N = _log(rng, 2, max(4, min(512, 268000000 // (E * K * 32)))) * 32
        T = _log(rng, 1, max(2, min(8192, 550000000000 // (k * K * N))))
        return dict(op=op, T=T, E=E, k=k, K=K, N=N, x=any_type(), out=any_type(),
                    swiglu=rng.random() < 0.5, spread=rng.choice([0.0, 1.0, 2.0]))
    E = _log(rng, 1, 256)
    k = rng.randint(1, min(E, 8))
    H = _log(rng, 8, 1024) * 8
    T = _log(rng, 1, max(2, min(16384, 67000000 // (k * H))))
    d = dict(op=op, T=T, E=E, k=k, H=H, x=any_type(), out=any_type(),
             drop=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "combine_bwd":
        return dict(d, rows=any_type(), renorm=rng.random() < 0.6)
    return dict(d, weights=rng.random() < 0.5)


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


def _routing(g, T, E, k, spread=0.0, drop=0.0):
    """Router logits and what routing makes of them: ids and both kinds of weights
    [T, k], the pairs by expert, each pair's row (-1: dropped), the experts' offsets."""
    crowd = -spread * torch.log(torch.arange(1, E + 1, device=DEV).float())
    logits = _randn(g, T, E) + crowd[torch.randperm(E, generator=g, device=DEV)]
    top, ids = torch.topk(logits, k, dim=1)
    order = torch.argsort(ids.reshape(-1), stable=True)
    kept = order
    if drop:
        keep = torch.ones(T * k, dtype=torch.bool, device=DEV)
        keep[torch.randperm(T * k, generator=g, device=DEV)[:int(drop * T * k)]] = False
        kept = order[keep[order]]
    pos = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    pos[kept] = torch.arange(kept.numel(), dtype=torch.int32, device=DEV)
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = counts.cumsum(0)
    return dict(logits=logits, ids=ids.int(), w=torch.softmax(top, 1),
                w_all=torch.softmax(logits, 1).gather(1, ids), sorted_pair=order.int(), pos=pos,
                kept=kept.numel(), offsets=off, host_offsets=off.tolist())


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "quant":
        E, R, K = case["E"], case["R"], case["K"]
        st["v"] = (0.02 * _activations(g, E * R, K, torch.float32)).view(E, R, K).to(
            TYPES[case["x"]])
    elif op == "product":
        E, K, N = case["E"], case["K"], case["N"]
        st["v"] = _activations(g, case["T"], K, TYPES[case["x"]])
        st.update(_routing(g, case["T"], E, case["k"], case["spread"]))
        blocks, scales = [], []
        for _ in range(E):  # one expert's matrix at a time, as a loader has them
            codes, e = _plain_blocks(0.02 * _randn(g, N, K))
            codes = codes.view(N, K)
            blocks.append(codes[:, 0::2] | (codes[:, 1::2] << 4))
            scales.append((e + 127).to(torch.uint8))
        st["blocks"], st["scales"] = torch.stack(blocks), torch.stack(scales)
    else:
        T, H = case["T"], case["H"]
        st.update(_routing(g, T, case["E"], case["k"], drop=case["drop"]))
        if op == "dispatch":
            st["v"] = _activations(g, T, H, TYPES[case["x"]])
        elif op == "combine":
            st["v"] = _randn(g, st["kept"], H).to(TYPES[case["x"]])
        else:
            st["dy"] = (0.01 * _randn(g, T, H)).to(TYPES[case["x"]])
            st["v"] = _randn(g, st["kept"], H).to(TYPES[case["rows"]])
    return st


# ---- the passes -----------------------------------------------------------

def run(st):
    return (_own if own else _plain)[st["op"]](st)


def _pow2(e):
    """fp32 2^e, to the bit, of whole e from -127 to 127 (exp2 is off by a rounding)."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).view(torch.float32)


def _plain_blocks(v):
    """fp32 [..., n] -> e2m1 codes (uint8 [..., n/32, 32]) and exponents (int [..., n/32])."""
    v = v.reshape(*v.shape[:-1], -1, BLOCK)
    top = v.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)
    a = v * _pow2(-e)[..., None]
    m = a.abs()
    codes = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
    codes = codes + (m >= 3.5) + (m > 5.0) + 8 * torch.signbit(a)
    return codes.to(torch.uint8), e


def _plain_values(v):
    """fp32 [..., n] -> what its blocks stand for."""
    codes, e = _plain_blocks(v)
    table = torch.tensor(E2M1, device=DEV)
    return (table[codes.int()] * _pow2(e)[..., None]).reshape(v.shape)


def _plain_quant(st):
    v = st["v"].float()
    if st["cols"]:
        v = v.transpose(1, 2).contiguous()
    return _plain_values(v).to(TYPES[st["out"]])


def _plain_stack(st, e):
    """Expert e's matrix as fp32 [N, K]."""
    c = st["blocks"][e]
    codes = torch.stack((c & 15, c >> 4), 2).view(c.shape[0], -1, BLOCK)
    v = torch.tensor(E2M1, device=DEV)[codes.int()]
    v = v * _pow2(st["scales"][e].int() - 127)[:, :, None]
    return v.view(c.shape[0], -1)


def _plain_product(st):
    a = _plain_values(st["v"].float())
    rows = a[st["sorted_pair"].long() // st["k"]]
    off = st["host_offsets"]
    # a product for each expert that has rows: they have different row counts
    out = torch.cat([rows[off[e]:off[e + 1]] @ _plain_stack(st, e).t()
                     for e in range(st["E"]) if off[e + 1] > off[e]])
    if st["swiglu"]:
        gate, up = out.chunk(2, dim=1)
        out = gate * torch.sigmoid(gate) * up
    return out.to(TYPES[st["out"]])


def _plain_dispatch(st):
    pos = st["pos"].long()
    pairs = torch.nonzero(pos >= 0).view(-1)
    src = torch.empty_like(pairs)
    src[pos[pairs]] = pairs
    rows = st["v"].float()[src // st["k"]]
    if st["weights"]:
        rows = rows * st["w"].view(-1)[src][:, None]
    return rows.to(TYPES[st["out"]])


def _plain_pairs(st):
    """Each pair's row, zeros for a dropped one: fp32 [T, k, H]."""
    pos = st["pos"].long()
    rows = st["v"].float()[pos.clamp(min=0)] * (pos >= 0)[:, None]
    return rows.view(st["T"], st["k"], -1)


def _plain_combine(st):
    rows = _plain_pairs(st)
    if st["weights"]:
        rows = rows * st["w"][:, :, None]
    return rows.sum(1).to(TYPES[st["out"]])


def _plain_combine_bwd(st):
    dy = st["dy"].float()
    w = st["w"] if st["renorm"] else st["w_all"]
    pos = st["pos"].long()
    dw = (dy[:, None, :] * _plain_pairs(st)).sum(2)
    drows = torch.empty_like(st["v"], dtype=torch.float32)
    drows[pos[pos >= 0]] = (w[:, :, None] * dy[:, None, :]).view(len(pos), -1)[pos >= 0]
    mean = (w * dw).sum(1, keepdim=True)
    ids = st["ids"].long()
    if st["renorm"]:
        dlogits = torch.zeros_like(st["logits"]).scatter(1, ids, w * (dw - mean))
    else:
        p = torch.softmax(st["logits"], 1)
        dlogits = p * (torch.zeros_like(p).scatter(1, ids, dw) - mean)
    return dict(drows=drows.to(TYPES[st["out"]]), dw=dw, dlogits=dlogits)


_plain = dict(quant=_plain_quant, product=_plain_product, dispatch=_plain_dispatch,
              combine=_plain_combine, combine_bwd=_plain_combine_bwd)


def _lib():
    from grouped_nf4_gemm_quantize_amd import binding

    return binding


def _own_quant(st):
    codes, scales = _lib().quantize_mxfp4(st["v"], transpose=st["cols"])
    return _lib().dequantize_mxfp4(codes, scales, dtype=TYPES[st["out"]])


def _own_product(st):
    return _lib().grouped_gemm_mx4(st["v"], None, st["blocks"], st["scales"], st["offsets"],
                                   st["T"] * st["k"], gather=st["sorted_pair"],
                                   gather_div=st["k"], swiglu=st["swiglu"],
                                   out_dtype=TYPES[st["out"]])


def _own_dispatch(st):
    return _lib().moe_dispatch(st["v"], st["pos"], st["k"], w=st["w"] if st["weights"] else None,
                               rows=st["kept"], out_dtype=TYPES[st["out"]])


def _own_combine(st):
    return _lib().moe_combine(st["v"], st["pos"], st["k"], w=st["w"] if st["weights"] else None,
                              y_dtype=TYPES[st["out"]])


def _own_combine_bwd(st):
    w = st["w"] if st["renorm"] else st["w_all"]
    drows, dw = _lib().moe_combine_backward(st["dy"], st["v"], st["pos"], st["k"], w=w,
                                            drows_dtype=TYPES[st["out"]])
    dlogits = _lib().moe_route_backward(st["logits"], st["ids"], dw, renormalize=st["renorm"])
    return dict(drows=drows, dw=dw, dlogits=dlogits)


_own = dict(quant=_own_quant, product=_own_product, dispatch=_own_dispatch,
            combine=_own_combine, combine_bwd=_own_combine_bwd)


# ---- what a pass cannot do without ----------------------------------------

def work(case):
    op = case["op"]
    if op == "quant":
        n = case["E"] * case["R"] * case["K"]
        # the values, and the 4-bit blocks written once and read once
        return dict(bytes=n * (BYTES[case["x"]] + BYTES[case["out"]]) + 2 * n * 17 // 32,
                    flops=4 * n)
    k, E = case["k"], case["E"]
    P = case["T"] * k
    if op == "product":
        K, N = case["K"], case["N"]
        # the experts that a uniform routing hits
        hit = E * (1 - (1 - k / E) ** case["T"])
        b = hit * N * K * 17 / 32 + case["T"] * K * BYTES[case["x"]] + 4 * P
        n_out = N // 2 if case["swiglu"] else N
        return dict(bytes=b + P * n_out * BYTES[case["out"]], flops=2 * P * N * K)
    T, H = case["T"], case["H"]
    R = P - int(case["drop"] * P)
    xb, ob = BYTES[case["x"]], BYTES[case["out"]]
    if op == "dispatch":
        return dict(bytes=T * H * xb + R * H * ob + 4 * P * (2 if case["weights"] else 1),
                    flops=R * H)
    if op == "combine":
        return dict(bytes=R * H * xb + T * H * ob + 4 * P * (2 if case["weights"] else 1),
                    flops=2 * R * H)
    return dict(bytes=T * H * xb + R * H * (BYTES[case["rows"]] + ob) + 16 * P + 8 * T * E,
                flops=3 * R * H + 4 * T * E)


# ---- the definitions in 64 bits -------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f8 = torch.float64

    def blocked(v):
        """What MXFP4 blocks along the last axis stand for, by steps of the e2m1 grid."""
        b = v.to(f8).reshape(-1, BLOCK)
        top = b.abs().max(1, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 2
        e = torch.where(top > 0, e, 0 * e - 127).clamp(min=-127)
        unit = ((e.long() + 1023) << 52).view(f8)
        q = (b / unit).abs()
        step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0)).to(f8)
        q = (torch.round(q / step) * step).clamp(max=6.0)
        return (torch.copysign(q, b) * unit).reshape(v.shape)

    if op == "quant":
        v = st["v"]
        return blocked(v.transpose(1, 2).contiguous() if case["cols"] else v)
    k, T = case["k"], case["T"]
    if op == "product":
        a = blocked(st["v"])
        grid = torch.tensor(E2M1, dtype=f8, device=DEV)
        parts = []
        for e in range(case["E"]):
            pairs = torch.nonzero(st["ids"].reshape(-1) == e).view(-1)
            if not pairs.numel():
                continue
            x = a[torch.div(pairs, k, rounding_mode="floor")]
            s = ((st["scales"][e].long() + (1023 - 127)) << 52).view(f8)
            s = s.repeat_interleave(BLOCK // 2, 1)
            b = st["blocks"][e].int()
            parts.append(x[:, 0::2] @ (grid[b % 16] * s).t() + x[:, 1::2] @ (grid[b // 16] * s).t())
        y = torch.cat(parts)
        if case["swiglu"]:
            n = y.shape[1] // 2
            y = y[:, :n] / (1 + torch.exp(-y[:, :n])) * y[:, n:]
        return y
    pos = st["pos"].long()
    kept = pos >= 0
    pairs = torch.nonzero(kept).view(-1)
    pairs = pairs[torch.argsort(pos[pairs])]  # the pair of each row
    tok = torch.div(pairs, k, rounding_mode="floor")
    v = st["v"].to(f8)
    if op == "dispatch":
        return v[tok] * st["w"].reshape(-1)[pairs].to(f8)[:, None] if case["weights"] else v[tok]
    if op == "combine":
        if case["weights"]:
            v = v * st["w"].reshape(-1)[pairs].to(f8)[:, None]
        return torch.zeros(T, case["H"], dtype=f8, device=DEV).index_add_(0, tok, v)
    # by differentiating the definition, a slot of every token at a time
    dy = st["dy"].to(f8)
    logits = st["logits"].to(f8).requires_grad_()
    ids = st["ids"].long()
    if case["renorm"]:
        w = torch.softmax(torch.gather(logits, 1, ids), 1)
    else:
        w = torch.gather(torch.softmax(logits, 1), 1, ids)
    dw = torch.zeros(T * k, dtype=f8, device=DEV)
    dw[pairs] = torch.cat([(dy[tok[i:i + 8192]] * v[i:i + 8192]).sum(1)
                           for i in range(0, len(pairs), 8192)])
    dw = dw.view(T, k)
    (dlogits,) = torch.autograd.grad(w, logits, dw)
    drows = dy[tok] * w.detach().reshape(-1)[pairs][:, None]
    return dict(drows=drows, dw=dw, dlogits=dlogits)
