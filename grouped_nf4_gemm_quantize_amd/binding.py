"""ctypes binding of libnf4moe.so (the C ABI in include/nf4moe.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their pointers and the current HIP stream are passed to the C
entry points, and a non-zero status becomes an exception carrying the
library's message.  PyTorch supplies device memory and streams; every step of
the computation runs in the library's HIP kernels.  If the shared library is
missing, every call raises -- there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnf4moe.so")

F32, BF16, F16 = 0, 1, 2
NOALLOC_SCRATCH_BYTES = 32 << 20  # NF4MOE_NOALLOC_SCRATCH_BYTES
EPI_NONE, EPI_SWIGLU, EPI_SWIGLU_BWD = 0, 1, 2

STATUS = {
    0: "NF4MOE_OK", -1: "NF4MOE_EINVAL", -2: "NF4MOE_ESHAPE", -3: "NF4MOE_EBLOCK",
    -4: "NF4MOE_ETOPK", -5: "NF4MOE_EDTYPE", -6: "NF4MOE_EWORKSPACE",
    -7: "NF4MOE_EOVERFLOW", -8: "NF4MOE_EHIP",
}


class Nf4MoeError(RuntimeError):
    """A library call returned a negative status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class LoraStruct(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("r", ctypes.c_int),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class MuonTensorStruct(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("m_out", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("w_out", ctypes.c_void_p), ("w16", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("E", ctypes.c_int), ("r", ctypes.c_int),
                ("rank_major", ctypes.c_int), ("w_dtype", ctypes.c_int),
                ("w16_dtype", ctypes.c_int), ("scale", ctypes.c_double)]


_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_vp = ctypes.c_void_p
_c_size = ctypes.c_size_t
_c_f32 = ctypes.c_float
_c_f64 = ctypes.c_double

_DGRAD_ARGS = [_c_vp, _c_int, _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_i64,
               _c_i64, _c_i64, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_vp]
_BACKWARD_ARGS = [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_int,
                  _c_int, _c_vp, _c_vp, _c_vp, _c_vp, ctypes.POINTER(LoraStruct),
                  ctypes.POINTER(LoraStruct), _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_vp,
                  _c_vp, _c_size, _c_vp]

_SIGNATURES = {
    "nf4moe_strerror": (ctypes.c_char_p, [_c_int]),
    "nf4moe_last_error": (ctypes.c_char_p, []),
    "nf4moe_version": (ctypes.c_char_p, []),
    "nf4moe_codebook": (_c_int, [ctypes.POINTER(ctypes.c_float)]),
    "nf4moe_packed_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64]),
    "nf4_quantize_experts": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int,
                                      _c_vp, _c_vp, _c_vp, _c_vp]),
    "nf4moe_f16_range_check": (_c_int, [_c_vp, _c_int, _c_i64, _c_vp, _c_vp]),
    "moe_route_permute_workspace": (_c_size, [_c_i64, _c_int, _c_int]),
    "moe_route_permute": (_c_int, [_c_vp, _c_i64, _c_int, _c_int, _c_int, _c_vp, _c_vp,
                                   _c_vp, _c_vp, _c_vp, _c_vp, _c_size, _c_vp]),
    "grouped_nf4_gemm": (_c_int, [_c_vp, _c_int, _c_i64, _c_vp, _c_int, _c_vp, _c_vp,
                                  _c_vp, _c_int, _c_i64, _c_i64, _c_i64,
                                  ctypes.POINTER(LoraStruct), _c_int, _c_vp, _c_vp,
                                  _c_vp, _c_int, _c_vp]),
    "moe_expert_forward_workspace": (_c_size, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "moe_expert_forward": (_c_int, [_c_vp, _c_int, _c_vp, _c_i64, _c_int, _c_int, _c_int,
                                    _c_int, _c_int, _c_vp, _c_vp, _c_vp, _c_vp,
                                    ctypes.POINTER(LoraStruct), ctypes.POINTER(LoraStruct),
                                    _c_vp, _c_int, _c_vp, _c_size, _c_vp]),
    "moe_expert_forward_noalloc": (_c_int, [_c_vp, _c_int, _c_vp, _c_i64, _c_int, _c_int, _c_int,
                                            _c_int, _c_int, _c_vp, _c_vp, _c_vp, _c_vp,
                                            ctypes.POINTER(LoraStruct),
                                            ctypes.POINTER(LoraStruct), _c_vp, _c_int, _c_vp]),
    "moe_expert_forward_routing": (_c_int, [_c_vp, _c_i64, _c_int, _c_int, _c_int, _c_int,
                                            ctypes.POINTER(_c_vp), ctypes.POINTER(_c_vp),
                                            ctypes.POINTER(_c_vp), ctypes.POINTER(_c_vp)]),
    "nbit_codebook": (_c_int, [_c_int, ctypes.POINTER(ctypes.c_float)]),
    "nbit_quantize_experts": (_c_int, [_c_int, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int,
                                       _c_vp, _c_vp, _c_vp, _c_vp]),
    "grouped_nbit_gemm": (_c_int, [_c_int, _c_vp, _c_int, _c_i64, _c_vp, _c_int, _c_vp, _c_vp,
                                   _c_vp, _c_int, _c_i64, _c_i64, _c_i64,
                                   ctypes.POINTER(LoraStruct), _c_int, _c_vp, _c_vp,
                                   _c_vp, _c_int, _c_vp]),
    "moe_expert_forward_nbit": (_c_int, [_c_int, _c_vp, _c_int, _c_vp, _c_i64, _c_int, _c_int,
                                         _c_int, _c_int, _c_int, _c_vp, _c_vp, _c_vp, _c_vp,
                                         ctypes.POINTER(LoraStruct), ctypes.POINTER(LoraStruct),
                                         _c_vp, _c_int, _c_vp, _c_size, _c_vp]),
    "grouped_nf4_gemm_swiglu_bwd": (_c_int, [_c_vp, _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp,
                                             _c_int, _c_i64, _c_i64, _c_i64,
                                             ctypes.POINTER(LoraStruct), _c_vp, _c_vp, _c_vp,
                                             _c_vp]),
    "grouped_nf4_gemm_dgrad": (_c_int, _DGRAD_ARGS),
    "grouped_nbit_gemm_dgrad": (_c_int, [_c_int] + _DGRAD_ARGS),
    "moe_expert_backward_workspace": (_c_size, [_c_i64, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "moe_expert_backward": (_c_int, _BACKWARD_ARGS),
    "moe_expert_backward_nbit": (_c_int, [_c_int] + _BACKWARD_ARGS),
    "grouped_mxfp4_gemm": (_c_int, [_c_vp, _c_int, _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp,
                                    _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_vp,
                                    _c_int, _c_vp]),
    "moe_expert_forward_mxfp4": (_c_int, [_c_vp, _c_int, _c_vp, _c_i64, _c_int, _c_int, _c_int,
                                          _c_int, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                                          _c_int, _c_vp, _c_size, _c_vp]),
    "nbit_matvec": (_c_int, [_c_int, _c_vp, _c_int, _c_i64, _c_vp, _c_vp, _c_int, _c_vp, _c_int,
                             _c_i64, _c_i64, _c_vp, _c_vp, _c_int, _c_vp]),
    "block_norm_forward": (_c_int, [_c_vp, _c_int, _c_vp, _c_int, _c_vp, _c_int, _c_vp, _c_vp,
                                    _c_int, _c_f32, _c_f32, _c_f32, _c_f32, _c_i64, _c_i64,
                                    _c_vp, _c_vp, _c_int, _c_vp]),
    "block_norm_backward_workspace": (_c_size, [_c_i64, _c_i64]),
    "block_norm_backward": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_int, _c_vp,
                                     _c_int, _c_vp, _c_vp, _c_int, _c_f32, _c_f32, _c_f32,
                                     _c_f32, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                                     _c_vp, _c_size, _c_vp]),
    "lora_muon_step_workspace": (_c_size, [ctypes.POINTER(MuonTensorStruct), _c_int]),
    "lora_muon_step": (_c_int, [ctypes.POINTER(MuonTensorStruct), _c_int, _c_f64, _c_f64, _c_int,
                                _c_f64, _c_int, _c_f64, _c_f64, _c_f64, _c_f64, _c_vp, _c_size,
                                _c_vp]),
    "lora_orthogonalize_workspace": (_c_size, [_c_int, _c_int, _c_i64]),
    "lora_orthogonalize": (_c_int, [_c_vp, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_int, _c_f64,
                                    _c_f64, _c_f64, _c_f64, _c_vp, _c_int, _c_vp, _c_size,
                                    _c_vp]),
}

# storage modes of the nbit entry points (NF4MOE_QT_* in include/nf4moe.h)
QUANT_TYPES = {"nf4": 0, "fp4": 1, "int8": 3, "fp8": 4, "bf16": 5, "fp16": 6}
EIGHT_BIT = ("int8", "fp8")  # one byte per element: packed stacks are [E, N, K]
PASSTHROUGH = ("bf16", "fp16")  # the weights themselves, [E, N, K], no absmax
WHOLE = EIGHT_BIT + PASSTHROUGH  # one element per K position


def _qt(quant_type: str) -> int:
    if quant_type not in QUANT_TYPES:
        raise ValueError(f"unknown quant_type {quant_type!r} (one of {sorted(QUANT_TYPES)})")
    return QUANT_TYPES[quant_type]

_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m grouped_nf4_gemm_quantize_amd.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != 0:
        lib = load()
        msg = lib.nf4moe_last_error().decode()
        raise Nf4MoeError(status, msg or lib.nf4moe_strerror(status).decode())


# ------------------------------------------------------------ torch helpers

def _torch():
    import torch

    return torch


_dtype_codes: dict = {}


def _dtype_code(dt) -> int:
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
    code = _dtype_codes.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    return code


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(device=None) -> int:
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


def codebook(quant_type: str = "nf4"):
    """The 16 fp32 levels of a storage mode, by code (list of floats)."""
    lib = load()
    buf = (ctypes.c_float * 16)()
    if quant_type == "nf4":
        _check(lib.nf4moe_codebook(buf))
    else:
        _check(lib.nbit_codebook(_qt(quant_type), buf))
    return list(buf)


def packed_bytes(E: int, N: int, K: int) -> int:
    n = load().nf4moe_packed_bytes(E, N, K)
    if n < 0:
        _check(int(n))
    return int(n)


def quantize(w, nonfinite_flag=None, quant_type: str = "nf4"):
    """Quantise w [E, N, K] (fp32 or bf16, GPU) -> (packed u8, absmax f32).

    The passthrough modes return (the [E, N, K] bf16 / fp16 weights, None).
    """
    torch = _torch()
    if w.dim() != 3:
        raise ValueError("w must be [E, N, K]")
    E, N, K = w.shape
    if quant_type in PASSTHROUGH:
        dt = torch.bfloat16 if quant_type == "bf16" else torch.float16
        packed = torch.empty((E, N, K), dtype=dt, device=w.device)
        args = (_ptr(w), _dtype_code(w.dtype), E, N, K, 64, _ptr(packed), None,
                _ptr(nonfinite_flag), _stream(w.device))
        _check(load().nbit_quantize_experts(_qt(quant_type), *args))
        return packed, None
    per_byte = 1 if quant_type in EIGHT_BIT else 2
    packed = torch.empty((E, N, K // per_byte), dtype=torch.uint8, device=w.device)
    absmax = torch.empty((E, N, max(K // 64, 1)), dtype=torch.float32, device=w.device)
    args = (_ptr(w), _dtype_code(w.dtype), E, N, K, 64, _ptr(packed), _ptr(absmax),
            _ptr(nonfinite_flag), _stream(w.device))
    if quant_type == "nf4":
        _check(load().nf4_quantize_experts(*args))
    else:
        _check(load().nbit_quantize_experts(_qt(quant_type), *args))
    return packed, absmax


def f16_range_check(t, flags):
    """OR into ``flags`` (one int32 on the GPU) what an fp16 conversion of the
    bf16 / fp32 tensor ``t`` would lose (see nf4moe_f16_range_check)."""
    if not t.is_contiguous():
        raise ValueError("t must be contiguous")
    _check(load().nf4moe_f16_range_check(_ptr(t), _dtype_code(t.dtype), t.numel(), _ptr(flags),
                                         _stream(t.device)))
    return flags


def route_permute(logits, k: int, renormalize: bool = True):
    """Top-k routing and the expert-grouped pair permutation."""
    torch = _torch()
    T, E = logits.shape
    dev = logits.device
    P = T * k
    out = dict(
        ids=torch.empty((T, k), dtype=torch.int32, device=dev),
        w=torch.empty((T, k), dtype=torch.float32, device=dev),
        sorted_pair=torch.empty(P, dtype=torch.int32, device=dev),
        pair_pos=torch.empty(P, dtype=torch.int32, device=dev),
        offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
    )
    lib = load()
    ws_bytes = lib.moe_route_permute_workspace(T, E, k)
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _check(lib.moe_route_permute(_ptr(logits), T, E, k, int(bool(renormalize)),
                                 _ptr(out["ids"]), _ptr(out["w"]), _ptr(out["sorted_pair"]),
                                 _ptr(out["pair_pos"]), _ptr(out["offsets"]), _ptr(ws),
                                 ws_bytes, _stream(dev)))
    return out


def make_lora(A, B, scale: float):
    """LoRA struct for A [E, r, K], B [E, N, r] (bf16 or fp16 GPU tensors).

    The tensors must stay alive until the call that uses the struct returns.
    """
    if A is None:
        return None
    s = LoraStruct(_ptr(A), _ptr(B), int(A.shape[1]), float(scale), _dtype_code(A.dtype))
    return s


def grouped_gemm(a, packed, absmax, offsets, P: int, gather=None, gather_div: int = 1,
                 lora=None, swiglu: bool = False, row_scale=None, scatter=None,
                 out=None, out_dtype=None, out_rows: Optional[int] = None,
                 quant_type: str = "nf4"):
    """Grouped NF4 GEMM (see grouped_nf4_gemm in include/nf4moe.h).

    ``lora`` is ``(A, B, scale)`` or None.  Returns ``out``.
    """
    torch = _torch()
    E, N, K2 = packed.shape
    K = K2 if quant_type in WHOLE else K2 * 2
    n_out = N // 2 if swiglu else N
    if out is None:
        rows = out_rows if out_rows is not None else P
        out = torch.empty((rows, n_out), dtype=out_dtype or torch.float16, device=a.device)
    lib = load()
    ls = make_lora(*lora) if lora is not None else None
    args = (_ptr(a), _dtype_code(a.dtype), a.shape[0], _ptr(gather), gather_div, _ptr(packed),
            _ptr(absmax), _ptr(offsets), E, P, N, K,
            ctypes.byref(ls) if ls is not None else None, EPI_SWIGLU if swiglu else EPI_NONE,
            _ptr(row_scale), _ptr(scatter), _ptr(out), _dtype_code(out.dtype),
            _stream(a.device))
    if quant_type == "nf4":
        _check(lib.grouped_nf4_gemm(*args))
    else:
        _check(lib.grouped_nbit_gemm(_qt(quant_type), *args))
    return out


def grouped_gemm_swiglu_bwd(a, packed, absmax, offsets, P: int, dh, gather=None,
                            gather_div: int = 1, lora=None, out=None, h_out=None):
    """The gate_up GEMM recomputed with the SwiGLU backward as its epilogue
    (see grouped_nf4_gemm_swiglu_bwd in include/nf4moe.h): returns
    ``out`` = [dh * up * silu'(gate) | dh * silu(gate)], fp16 [P, N]; pass an
    fp16 ``h_out`` [P, N/2] to get h = silu(gate) * up as well."""
    torch = _torch()
    E, N, K2 = packed.shape
    if out is None:
        out = torch.empty((P, N), dtype=torch.float16, device=a.device)
    ls = make_lora(*lora) if lora is not None else None
    _check(load().grouped_nf4_gemm_swiglu_bwd(
        _ptr(a), a.shape[0], _ptr(gather), gather_div, _ptr(packed), _ptr(absmax),
        _ptr(offsets), E, P, N, K2 * 2, ctypes.byref(ls) if ls is not None else None, _ptr(dh),
        _ptr(out), _ptr(h_out), _stream(a.device)))
    return out


def forward_workspace_bytes(T: int, H: int, I: int, E: int, k: int, r: int = 0) -> int:
    """Workspace of moe_forward; ``r`` is the larger adapter rank (0: none)."""
    return int(load().moe_expert_forward_workspace(T, H, I, E, k, r))


def moe_forward(x, logits, k: int, gu_packed, gu_absmax, dn_packed, dn_absmax,
                gu_lora=None, dn_lora=None, renormalize: bool = True, y=None,
                y_dtype=None, workspace=None, quant_type: str = "nf4"):
    """Full routed-expert layer (see moe_expert_forward in include/nf4moe.h).

    ``gu_lora`` / ``dn_lora`` are ``(A, B, scale)`` or None.  ``workspace`` is an
    optional preallocated uint8 GPU tensor.  Returns ``y``.
    """
    torch = _torch()
    T, H = x.shape
    E = logits.shape[1]
    I = dn_packed.shape[2] * (1 if quant_type in WHOLE else 2)
    if y is None:
        y = torch.empty((T, H), dtype=y_dtype or torch.bfloat16, device=x.device)
    lib = load()
    r = max([l[0].shape[1] for l in (gu_lora, dn_lora) if l is not None and l[0] is not None],
            default=0)
    ws_bytes = lib.moe_expert_forward_workspace(T, H, I, E, k, r)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=x.device)
    ls_gu = make_lora(*gu_lora) if gu_lora is not None else None
    ls_dn = make_lora(*dn_lora) if dn_lora is not None else None
    args = (_ptr(x), _dtype_code(x.dtype), _ptr(logits), T, H, I, E, k, int(bool(renormalize)),
            _ptr(gu_packed), _ptr(gu_absmax), _ptr(dn_packed), _ptr(dn_absmax),
            ctypes.byref(ls_gu) if ls_gu is not None else None,
            ctypes.byref(ls_dn) if ls_dn is not None else None,
            _ptr(y), _dtype_code(y.dtype), _ptr(workspace), workspace.numel(),
            _stream(x.device))
    if quant_type == "nf4":
        _check(lib.moe_expert_forward(*args))
    else:
        _check(lib.moe_expert_forward_nbit(_qt(quant_type), *args))
    return y


def moe_forward_noalloc(x, logits, k: int, gu_packed, gu_absmax, dn_packed, dn_absmax,
                        gu_lora=None, dn_lora=None, renormalize: bool = True, y=None,
                        y_dtype=None):
    """The layer forward on the library's fixed per-device scratch memory
    (see moe_expert_forward_noalloc): no workspace argument, nothing
    allocated by the library.  Returns ``y``."""
    torch = _torch()
    T, H = x.shape
    E = logits.shape[1]
    I = dn_packed.shape[2] * 2
    if y is None:
        y = torch.empty((T, H), dtype=y_dtype or torch.bfloat16, device=x.device)
    ls_gu = make_lora(*gu_lora) if gu_lora is not None else None
    ls_dn = make_lora(*dn_lora) if dn_lora is not None else None
    _check(load().moe_expert_forward_noalloc(
        _ptr(x), _dtype_code(x.dtype), _ptr(logits), T, H, I, E, k, int(bool(renormalize)),
        _ptr(gu_packed), _ptr(gu_absmax), _ptr(dn_packed), _ptr(dn_absmax),
        ctypes.byref(ls_gu) if ls_gu is not None else None,
        ctypes.byref(ls_dn) if ls_dn is not None else None,
        _ptr(y), _dtype_code(y.dtype), _stream(x.device)))
    return y


def forward_routing(workspace, T: int, H: int, I: int, E: int, k: int):
    """Device pointers (ints) of the routing a forward left in its workspace."""
    ids, w, sp, off = _c_vp(), _c_vp(), _c_vp(), _c_vp()
    _check(load().moe_expert_forward_routing(_ptr(workspace), T, H, I, E, k,
                                             ctypes.byref(ids), ctypes.byref(w),
                                             ctypes.byref(sp), ctypes.byref(off)))
    return dict(ids=ids.value, w=w.value, sorted_pair=sp.value, offsets=off.value)


def grouped_dgrad(a, packed, absmax, offsets, P: int, gather=None, gather_div: int = 1,
                  g_pre=None, row_scale=None, scatter=None, out=None, out_dtype=None,
                  out_rows: Optional[int] = None, quant_type: str = "nf4"):
    """Grouped dgrad through the packed stack (see grouped_nf4_gemm_dgrad).

    ``g_pre`` (the forward's [gate | up] pre-activation rows) selects the
    SwiGLU-backward epilogue.  Returns ``out`` ([rows, K] or [rows, 2K]).
    """
    torch = _torch()
    E, N, K2 = packed.shape
    K = K2 * 2
    n_out = 2 * K if g_pre is not None else K
    if out is None:
        rows = out_rows if out_rows is not None else P
        out = torch.empty((rows, n_out), dtype=out_dtype or torch.float16, device=a.device)
    lib = load()
    args = (_ptr(a), _dtype_code(a.dtype), a.shape[0], _ptr(gather), gather_div, _ptr(packed),
            _ptr(absmax), _ptr(offsets), E, P, N, K,
            EPI_SWIGLU_BWD if g_pre is not None else EPI_NONE, _ptr(g_pre),
            _dtype_code(g_pre.dtype) if g_pre is not None else F16, _ptr(row_scale),
            _ptr(scatter), _ptr(out), _dtype_code(out.dtype), _stream(a.device))
    if quant_type == "nf4":
        _check(lib.grouped_nf4_gemm_dgrad(*args))
    else:
        _check(lib.grouped_nbit_gemm_dgrad(_qt(quant_type), *args))
    return out


def backward_workspace_bytes(T: int, H: int, I: int, E: int, k: int, r: int = 0) -> int:
    return int(load().moe_expert_backward_workspace(T, H, I, E, k, r))


def moe_backward(x, logits, dy, k: int, gu_packed, gu_absmax, dn_packed, dn_absmax,
                 gu_lora=None, dn_lora=None, renormalize: bool = True, dx=None,
                 dx_dtype=None, workspace=None, quant_type: str = "nf4"):
    """Layer backward (see moe_expert_backward in include/nf4moe.h).

    Returns ``(dx, grads)`` where ``grads`` holds ``dA_gu``/``dB_gu`` and
    ``dA_dn``/``dB_dn`` (fp32) for the adapters given.
    """
    torch = _torch()
    T, H = x.shape
    E = logits.shape[1]
    I = dn_packed.shape[2] * 2
    dev = x.device
    if dx is None:
        dx = torch.empty((T, H), dtype=dx_dtype or torch.bfloat16, device=dev)
    r = 0
    grads = {}
    if gu_lora is not None:
        r = int(gu_lora[0].shape[1])
        grads["dA_gu"] = torch.empty((E, r, H), dtype=torch.float32, device=dev)
        grads["dB_gu"] = torch.empty((E, 2 * I, r), dtype=torch.float32, device=dev)
    if dn_lora is not None:
        r = int(dn_lora[0].shape[1])
        grads["dA_dn"] = torch.empty((E, r, I), dtype=torch.float32, device=dev)
        grads["dB_dn"] = torch.empty((E, H, r), dtype=torch.float32, device=dev)
    lib = load()
    ws_bytes = lib.moe_expert_backward_workspace(T, H, I, E, k, r)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    ls_gu = make_lora(*gu_lora) if gu_lora is not None else None
    ls_dn = make_lora(*dn_lora) if dn_lora is not None else None
    args = (_ptr(x), _dtype_code(x.dtype), _ptr(logits), _ptr(dy), _dtype_code(dy.dtype), T, H,
            I, E, k, int(bool(renormalize)), _ptr(gu_packed), _ptr(gu_absmax), _ptr(dn_packed),
            _ptr(dn_absmax), ctypes.byref(ls_gu) if ls_gu is not None else None,
            ctypes.byref(ls_dn) if ls_dn is not None else None, _ptr(dx), _dtype_code(dx.dtype),
            _ptr(grads.get("dA_gu")), _ptr(grads.get("dB_gu")), _ptr(grads.get("dA_dn")),
            _ptr(grads.get("dB_dn")), _ptr(workspace), workspace.numel(), _stream(dev))
    if quant_type == "nf4":
        _check(lib.moe_expert_backward(*args))
    else:
        _check(lib.moe_expert_backward_nbit(_qt(quant_type), *args))
    return dx, grads


def grouped_gemm_mxfp4(a, blocks, scales, offsets, P: int, gather=None, gather_div: int = 1,
                       swiglu: bool = False, row_scale=None, scatter=None, out=None,
                       out_dtype=None, out_rows: Optional[int] = None):
    """Grouped GEMM on MXFP4 stacks (see grouped_mxfp4_gemm in include/nf4moe.h)."""
    torch = _torch()
    E, N, K2 = blocks.shape
    K = K2 * 2
    n_out = N // 2 if swiglu else N
    if out is None:
        rows = out_rows if out_rows is not None else P
        out = torch.empty((rows, n_out), dtype=out_dtype or torch.float16, device=a.device)
    _check(load().grouped_mxfp4_gemm(
        _ptr(a), _dtype_code(a.dtype), a.shape[0], _ptr(gather), gather_div, _ptr(blocks),
        _ptr(scales), _ptr(offsets), E, P, N, K, EPI_SWIGLU if swiglu else EPI_NONE,
        _ptr(row_scale), _ptr(scatter), _ptr(out), _dtype_code(out.dtype), _stream(a.device)))
    return out


def moe_forward_mxfp4(x, logits, k: int, gu_blocks, gu_scales, dn_blocks, dn_scales,
                      renormalize: bool = True, y=None, y_dtype=None, workspace=None):
    """Routed-expert layer on MXFP4 stacks (see moe_expert_forward_mxfp4)."""
    torch = _torch()
    T, H = x.shape
    E = logits.shape[1]
    I = dn_blocks.shape[2] * 2
    if y is None:
        y = torch.empty((T, H), dtype=y_dtype or torch.bfloat16, device=x.device)
    lib = load()
    ws_bytes = lib.moe_expert_forward_workspace(T, H, I, E, k, 0)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=x.device)
    _check(lib.moe_expert_forward_mxfp4(
        _ptr(x), _dtype_code(x.dtype), _ptr(logits), T, H, I, E, k, int(bool(renormalize)),
        _ptr(gu_blocks), _ptr(gu_scales), _ptr(dn_blocks), _ptr(dn_scales), _ptr(y),
        _dtype_code(y.dtype), _ptr(workspace), workspace.numel(), _stream(x.device)))
    return y


# ---- operators around the routed experts ------------------------------------

MATVEC_TYPES = {"nf4": 0, "fp4": 1, "int4": 2, "mxfp4": 7}
GATE_AXES = {"none": 0, "token": 1, "channel": 2}
NS_COEFFS = (3.4445, -4.7750, 2.0315)


def _need(t, what: str, dev, shape=None, dtype=None):
    """A contiguous GPU tensor on ``dev`` of the given shape and type: its pointer."""
    if t.device != dev:
        raise ValueError(f"{what} is on {t.device}, not on {dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must be {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        return _ptr(t)  # raises
    return t.data_ptr()


def _call(dev, fn, *args) -> None:
    """One C call on the current stream of ``dev``, which is made the current
    device for it if it is not."""
    cuda = _torch().cuda
    if cuda.current_device() == dev.index:
        status = fn(*args, _raw_stream(dev.index))
    else:
        with cuda.device(dev):
            status = fn(*args, _raw_stream(dev.index))
    if status != 0:
        _check(status)


def _workspace(given, need: int, dev):
    """The caller's workspace, or a new one of ``need`` bytes (None for 0)."""
    if given is not None or need == 0:
        return given
    torch = _torch()
    return torch.empty(need, dtype=torch.uint8, device=dev)


def _span(workspace, dev):
    """Pointer and bytes of a workspace that may be None."""
    if workspace is None:
        return None, 0
    return _need(workspace, "workspace", dev), workspace.numel() * workspace.element_size()


def _raw_stream(index: int) -> int:
    """The handle of the current stream.  torch's own accessor for launchers costs 0.1 us,
    a Stream object 1.8 us of the 10 us that a small call takes on the host."""
    torch = _torch()
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(index) if get is not None else torch.cuda.current_stream(index).cuda_stream


def nbit_matvec(x, codes, scales, quant_type: str = "nf4", group: Optional[int] = None,
                zeros=None, bias=None, out=None, out_dtype=None):
    """A few rows times one 4-bit matrix: x [T, K] -> [T, N] (see nbit_matvec in
    include/nf4moe.h).

    ``codes`` is uint8 [N, K/2] and ``scales`` [N, K/group]: fp32 for ``"nf4"`` and
    ``"fp4"`` (what ``quantize`` returns, one expert's slice of it), fp32 / bf16 /
    fp16 for ``"int4"`` (``zeros`` uint8 [N, K/group], None: 8), e8m0 bytes for
    ``"mxfp4"``.  ``bias`` is fp32 [N].  ``group`` defaults to 64 (32 for mxfp4).  ``x`` is bf16 or
    fp16; bf16 x becomes fp16 for ``"nf4"`` and ``"int4"``.  int4 codes are made by the caller.
    """
    torch = _torch()
    if quant_type not in MATVEC_TYPES:
        raise ValueError(f"unknown quant_type {quant_type!r} (one of {sorted(MATVEC_TYPES)})")
    if x.dim() != 2 or codes.dim() != 2:
        raise ValueError("x must be [T, K] and codes [N, K/2]")
    dev = x.device
    T, K = x.shape
    N = codes.shape[0]
    if group is None:
        group = 32 if quant_type == "mxfp4" else 64
    if group < 1 or K % group:
        raise ValueError(f"K={K} is not a multiple of the group {group}")
    groups = (N, K // group)
    mx = quant_type == "mxfp4"
    if out is None:
        out = torch.empty(T, N, dtype=out_dtype or x.dtype, device=dev)
    _call(dev, load().nbit_matvec, MATVEC_TYPES[quant_type], _ptr(x), _dtype_code(x.dtype), T,
          _need(codes, "codes", dev, (N, K // 2), torch.uint8),
          _need(scales, "scales", dev, groups, torch.uint8 if mx else None),
          F32 if mx else _dtype_code(scales.dtype),
          None if zeros is None else _need(zeros, "zeros", dev, groups, torch.uint8), group, N, K,
          None if bias is None else _need(bias, "bias", dev, (N,), torch.float32),
          _need(out, "out", dev, (T, N)), _dtype_code(out.dtype))
    return out


def _norm_args(res, y, gate, gate_axis, w_pre, w_post, w_offset, alpha, beta, eps):
    """The arguments both directions of block_norm share, checked; from y to H."""
    torch = _torch()
    if res.dim() != 2:
        raise ValueError("the residual must be [T, H]")
    dev = res.device
    T, H = res.shape
    axis = "none" if gate is None else gate_axis
    if axis not in GATE_AXES:
        raise ValueError(f"unknown gate_axis {gate_axis!r} (one of {sorted(GATE_AXES)})")
    w = w_pre if w_pre is not None else w_post
    wt = w.dtype if w is not None else torch.float32
    return (None if y is None else _need(y, "y", dev, (T, H)),
            F32 if y is None else _dtype_code(y.dtype),
            None if gate is None else _need(gate, "gate", dev, (H if axis == "channel" else T,),
                                            torch.float32),
            GATE_AXES[axis],
            None if w_pre is None else _need(w_pre, "w_pre", dev, (H,), wt),
            None if w_post is None else _need(w_post, "w_post", dev, (H,), wt),
            _dtype_code(wt), w_offset, alpha, beta, eps, T, H)


def block_norm(residual, y=None, w_pre=None, w_post=None, gate=None, gate_axis: str = "token",
               alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6, w_offset: float = 0.0,
               r_out=None, h=None, h_dtype=None):
    """The norms after and before a block with its gate and residual scale (see
    block_norm_forward in include/nf4moe.h): returns ``(r, h)`` with
    r = beta * residual + alpha * gate * norm(y; w_post), h = norm(r; w_pre).

    Without ``y``, r is ``residual`` itself; without ``w_pre``, h is None; without
    ``w_post``, y is added as it is.  ``gate`` is fp32 [T] (``gate_axis="token"``) or
    [H] (``"channel"``).  ``r_out`` may be ``residual``.
    """
    torch = _torch()
    dev = residual.device
    args = _norm_args(residual, y, gate, gate_axis, w_pre, w_post, w_offset, alpha, beta, eps)
    if y is not None and r_out is None:
        r_out = torch.empty_like(residual)
    if w_pre is not None and h is None:
        h = torch.empty_like(residual, dtype=h_dtype or residual.dtype)
    _call(dev, load().block_norm_forward, _ptr(residual), _dtype_code(residual.dtype), *args,
          None if r_out is None else _need(r_out, "r_out", dev, residual.shape, residual.dtype),
          None if h is None else _need(h, "h", dev, residual.shape),
          F32 if h is None else _dtype_code(h.dtype))
    return (residual if y is None else r_out), h


def block_norm_backward(dh, d_r_out, r, y=None, w_pre=None, w_post=None, gate=None,
                        gate_axis: str = "token", alpha: float = 1.0, beta: float = 1.0,
                        eps: float = 1e-6, w_offset: float = 0.0, workspace=None,
                        dresidual=None, dy=None):
    """Gradients of ``block_norm`` (see block_norm_backward in include/nf4moe.h) from
    those of h (None exactly where ``w_pre`` is) and r (None where nothing reaches it but
    through h); ``r`` is what the forward returned.

    Returns a dict with ``dresidual`` and, where their inputs are given, ``dy``,
    ``dgate``, ``dw_pre`` and ``dw_post`` (the last three fp32).  ``dresidual=`` may name
    ``d_r_out`` and ``dy=`` may name ``y`` or ``dh`` (of y's type) as the place to write to.
    """
    torch = _torch()
    dev = r.device
    args = _norm_args(r, y, gate, gate_axis, w_pre, w_post, w_offset, alpha, beta, eps)
    T, H = r.shape
    if dresidual is None:
        dresidual = torch.empty_like(r)
    else:
        _need(dresidual, "dresidual", dev, r.shape, r.dtype)
    out = dict(dresidual=dresidual)
    if y is not None:
        out["dy"] = torch.empty_like(y) if dy is None else dy
        if dy is not None:
            _need(dy, "dy", dev, y.shape, y.dtype)
    elif dy is not None:
        raise ValueError("dy is written only where y is given")
    if gate is not None:
        out["dgate"] = torch.empty_like(gate)
    if w_pre is not None:
        out["dw_pre"] = torch.empty_like(w_pre, dtype=torch.float32)
    if w_post is not None:
        out["dw_post"] = torch.empty_like(w_post, dtype=torch.float32)
    ws = _workspace(workspace, load().block_norm_backward_workspace(T, H), dev)
    ptr = lambda k: out[k].data_ptr() if k in out else None  # noqa: E731
    _call(dev, load().block_norm_backward,
          None if dh is None else _need(dh, "dh", dev, r.shape),
          F32 if dh is None else _dtype_code(dh.dtype),
          None if d_r_out is None else _need(d_r_out, "d_r_out", dev, r.shape, r.dtype),
          _ptr(r), _dtype_code(r.dtype), *args, ptr("dresidual"), ptr("dy"), ptr("dgate"),
          ptr("dw_pre"), ptr("dw_post"), *_span(ws, dev))
    return out


def lora_orthogonalize(u, rank_major: bool = True, steps: int = 5, coeffs=NS_COEFFS,
                       eps: float = 1e-7, out=None, out_dtype=None, workspace=None):
    """Newton-Schulz orthogonalisation of per-expert factors u [E, r, n] (or
    [E, n, r] with ``rank_major=False``); see lora_orthogonalize in include/nf4moe.h."""
    torch = _torch()
    if u.dim() != 3:
        raise ValueError("u must be [E, r, n] or [E, n, r]")
    dev = u.device
    E, r, n = u.shape if rank_major else (u.shape[0], u.shape[2], u.shape[1])
    if out is None:
        out = torch.empty(u.shape, dtype=out_dtype or u.dtype, device=dev)
    lib = load()
    ws = _workspace(workspace, lib.lora_orthogonalize_workspace(E, r, n), dev)
    _call(dev, lib.lora_orthogonalize, _ptr(u), _dtype_code(u.dtype), E, r, n,
          int(bool(rank_major)), steps, *coeffs, eps, _need(out, "out", dev, u.shape),
          _dtype_code(out.dtype), *_span(ws, dev))
    return out


def lora_muon_step(tensors, lr: float, momentum: float = 0.95, nesterov: bool = True,
                   weight_decay: float = 0.0, steps: int = 5, coeffs=NS_COEFFS,
                   eps: float = 1e-7, workspace=None) -> None:
    """One optimiser step of up to eight adapter tensors (see lora_muon_step in
    include/nf4moe.h), in place unless other outputs are named.

    Each of ``tensors`` is a dict with ``grad`` and ``momentum`` (fp32), ``w`` (fp32,
    bf16 or fp16), all [E, r, n] (``rank_major=True``, the A factors) or [E, n, r]
    (False, the B factors), and optionally ``scale`` (of the update, default 1),
    ``momentum_out``, ``w_out`` and ``w16`` (a bf16 or fp16 copy of the new w).
    """
    torch = _torch()
    if not 1 <= len(tensors) <= 8:
        raise ValueError(f"1 to 8 tensors are taken, got {len(tensors)}")
    arr = (MuonTensorStruct * len(tensors))()
    dev = tensors[0]["grad"].device
    for s, t in zip(arr, tensors):
        g, w, rank_major = t["grad"], t["w"], bool(t["rank_major"])
        if g.dim() != 3:
            raise ValueError("grad must be [E, r, n] or [E, n, r]")
        shape, m = g.shape, t["momentum"]
        w16 = t.get("w16")
        m_out, w_out = t.get("momentum_out"), t.get("w_out")
        s.grad = _need(g, "grad", dev, shape, torch.float32)
        s.m = _need(m, "momentum", dev, shape, torch.float32)
        s.m_out = s.m if m_out is None else _need(m_out, "momentum_out", dev, shape, torch.float32)
        s.w = _need(w, "w", dev, shape)
        s.w_out = s.w if w_out is None else _need(w_out, "w_out", dev, shape, w.dtype)
        s.w_dtype = _dtype_code(w.dtype)
        if w16 is not None:
            s.w16 = _need(w16, "w16", dev, shape)
            s.w16_dtype = _dtype_code(w16.dtype)
        s.E, s.r, s.n = shape if rank_major else (shape[0], shape[2], shape[1])
        s.rank_major = int(rank_major)
        s.scale = t.get("scale", 1.0)
    lib = load()
    ws = _workspace(workspace, lib.lora_muon_step_workspace(arr, len(arr)), dev)
    _call(dev, lib.lora_muon_step, arr, len(arr), lr, momentum, int(bool(nesterov)), weight_decay,
          steps, *coeffs, eps, *_span(ws, dev))
