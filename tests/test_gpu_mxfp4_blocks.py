"""MXFP4 blocks on the GPU, byte for byte against the format's rule in 64 bits.  No
tolerance: every quotient by a power of two is exact, so the nearest code is one code."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
TT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def host(t):
    return t.detach().double().cpu().numpy()


def bytes_of(lib, x, **kw):
    c, s = lib.quantize_mxfp4(x, **kw)
    return c.cpu().numpy(), s.cpu().numpy()


def same(lib, x, transpose=False):
    c, s = bytes_of(lib, x, transpose=transpose)
    v = host(x)
    want, scales = oracle.quantize_mxfp4(np.swapaxes(v, -1, -2) if transpose else v)
    assert s.shape == scales.shape and np.array_equal(s, scales), np.argwhere(s != scales)[:4]
    assert c.shape == want.shape and np.array_equal(c, want), np.argwhere(c != want)[:4]


def every_16(t):
    """Every 16-bit value beside a largest one of each nearby exponent."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(t)
    v = bits[torch.isfinite(bits.float())].float()
    rows = []
    for up in (0, 1, 3):
        top = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1e-40))) + up) * 1.5
        top = top.clamp(max=torch.finfo(t).max).to(t)
        rows.append(torch.stack([v.to(t), top], 1).repeat(1, 16))
    return torch.cat(rows).to(DEV)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("transpose", [False, True])
def test_every_16_bit_value(gpu_lib, t, transpose):
    x = every_16(TT[t])
    x = x.t().contiguous() if transpose else x
    same(gpu_lib, x, transpose)


@pytest.mark.parametrize("transpose", [False, True])
def test_fp32_of_every_exponent(gpu_lib, transpose):
    rng = np.random.default_rng(0)
    bits = rng.integers(0, 1 << 32, (3000, 32), dtype=np.uint32)
    # exponents near each other, over the whole range, subnormals among them
    e = np.clip(rng.integers(0, 255, (3000, 1)) + rng.integers(-4, 1, (3000, 32)), 0, 254)
    x = ((bits & 0x807fffff) | (e.astype(np.uint32) << 23)).view(np.float32)
    x[::7] = np.round(x[::7].astype(np.float64) / 2.0 ** (e[::7, :1] - 130.0)).astype(np.float32)
    x = torch.from_numpy(x).to(DEV)
    same(gpu_lib, x.t().contiguous() if transpose else x, transpose)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("transpose", [False, True])
def test_ties_and_signed_zeros(gpu_lib, t, transpose):
    v = torch.arange(-64, 64).float() * 0.125  # every eighth up to 8, ties among them
    x = v.repeat(32, 1) * 2.0 ** torch.arange(-12, 4).repeat(2)[:, None]
    x[:, 1::32] = -0.0
    x = x.to(TT[t]).to(DEV)
    same(gpu_lib, x.t().contiguous() if transpose else x, transpose)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("transpose", [False, True])
def test_blocks_without_a_value(gpu_lib, t, transpose):
    x = torch.randn(6, 128, generator=torch.Generator().manual_seed(1))
    x[0, 5], x[1, 40], x[2, 70] = float("inf"), float("-inf"), float("nan")
    x[3, 31], x[3, 32] = float("nan"), float("inf")
    x[4, 96:] = 0.0
    x[5, :32] = -0.0
    x = x.to(TT[t]).to(DEV)
    same(gpu_lib, x.t().contiguous() if transpose else x, transpose)
    c, s = gpu_lib.quantize_mxfp4(x)
    back = gpu_lib.dequantize_mxfp4(c, s, torch.float32)
    bad = ~torch.isfinite(x.float()).view(6, 4, 32).all(2)
    assert torch.equal(torch.isnan(back).view(6, 4, 32).all(2), bad)
    assert torch.equal(torch.isnan(back).view(6, 4, 32).any(2), bad)


SHAPES = [(1, 32), (1, 2048), (3, 96), (77, 2880), (1000, 32), (5, 16384), (2049, 160)]


@pytest.mark.parametrize("R,K", SHAPES)
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_rows(gpu_lib, t, R, K):
    x = torch.randn(R, K, device=DEV, generator=torch.Generator(DEV).manual_seed(R + K)).to(TT[t])
    same(gpu_lib, x)


@pytest.mark.parametrize("E,R,K", [(1, 32, 1), (1, 64, 3), (2, 96, 65), (1, 32, 64), (3, 160, 130),
                                   (1, 2048, 31), (2, 288, 257), (1, 4128, 128), (5, 256, 96)])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_columns_of_stacks(gpu_lib, t, E, R, K):
    x = torch.randn(E, R, K, device=DEV, generator=torch.Generator(DEV).manual_seed(E + R + K))
    same(gpu_lib, x.to(TT[t]), True)


def test_a_stack_is_its_experts(gpu_lib):
    x = torch.randn(3, 40, 96, device=DEV, dtype=torch.bfloat16)
    same(gpu_lib, x)
    c, s = gpu_lib.quantize_mxfp4(x)
    ci, si = gpu_lib.quantize_mxfp4(x[1])
    assert torch.equal(c[1], ci) and torch.equal(s[1], si)


@pytest.mark.parametrize("offset", [1, 3])
def test_columns_at_any_element(gpu_lib, offset):
    flat = torch.randn(offset + 64 * 33, device=DEV).to(torch.bfloat16)
    x = flat[offset:].view(64, 33)
    same(gpu_lib, x, True)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_every_code_and_scale_reads_back(gpu_lib, t):
    b = np.arange(256, dtype=np.uint8)
    codes = np.tile(b.reshape(16, 16), (256, 1))  # [4096, 16] bytes: every pair of codes
    scales = np.repeat(b, 16)[:, None]
    got = gpu_lib.dequantize_mxfp4(torch.from_numpy(codes).to(DEV),
                                   torch.from_numpy(scales.copy()).to(DEV), TT[t])
    with np.errstate(over="ignore"):
        want = torch.from_numpy(oracle.dequantize_mxfp4(codes, scales)).to(TT[t])
    got = got.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    at = ~torch.isnan(want)
    assert torch.equal(got[at], want[at])
    assert torch.equal(torch.signbit(got[at]), torch.signbit(want[at]))


@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (1, 2048), (333, 2880)])
def test_reading_back_sizes_and_neighbours(gpu_lib, R, K):
    g = torch.Generator(DEV).manual_seed(R)
    x = torch.randn(R, K, device=DEV, generator=g)
    c, s = gpu_lib.quantize_mxfp4(x)
    out = torch.full((R + 2, K), 7.0, device=DEV, dtype=torch.float16)
    gpu_lib.dequantize_mxfp4(c, s, out=out[1:R + 1])
    want = oracle.dequantize_mxfp4(c.cpu().numpy(), s.cpu().numpy())
    assert np.array_equal(host(out[1:R + 1]), want)  # exact: fp16 holds these
    assert (out[0] == 7).all() and (out[-1] == 7).all()


def test_outputs_are_the_callers_and_neighbours_stay(gpu_lib):
    x = torch.randn(64, 96, device=DEV)
    for tr in (False, True):
        n, m = (96, 64) if tr else (64, 96)
        c = torch.full((n + 2, m // 2), 9, dtype=torch.uint8, device=DEV)
        s = torch.full((n + 2, m // 32), 9, dtype=torch.uint8, device=DEV)
        got = gpu_lib.quantize_mxfp4(x, transpose=tr, codes=c[1:-1], scales=s[1:-1])
        want = gpu_lib.quantize_mxfp4(x, transpose=tr)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (c[0] == 9).all() and (c[-1] == 9).all() and (s[0] == 9).all() and (s[-1] == 9).all()


def test_refusals_of_the_binding(gpu_lib):
    x = torch.randn(32, 64, device=DEV)
    with pytest.raises(ValueError):
        gpu_lib.quantize_mxfp4(x[:, :48])
    with pytest.raises(ValueError):
        gpu_lib.quantize_mxfp4(x[:31], transpose=True)
    with pytest.raises(ValueError):
        gpu_lib.quantize_mxfp4(x.t())  # not contiguous
    with pytest.raises(TypeError):
        gpu_lib.quantize_mxfp4(x.double())
    c, s = gpu_lib.quantize_mxfp4(x)
    with pytest.raises(ValueError):
        gpu_lib.dequantize_mxfp4(c, s[:, :1])
    with pytest.raises(TypeError):
        gpu_lib.dequantize_mxfp4(c.int(), s)
    with pytest.raises(ValueError):
        gpu_lib.dequantize_mxfp4(c.cpu(), s)
