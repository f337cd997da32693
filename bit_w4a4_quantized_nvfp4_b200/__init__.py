"""B200 (sm_100a) SVDQuant W4A4 and AWQ W4A16 linear layers, with the 8-bit
(E4M3) linear layer and the rotary positions that stand beside them.

A thin ctypes binding over ``libsvdq.so`` (C ABI in ``include/svdq.h``).
Every function here only marshals arguments: torch tensors provide device
memory and the current CUDA stream, and every step of the layer runs in the
library's kernels. There is no CPU fallback: importing works without a GPU,
but calling an entry point without the built library raises.

The layer (blog "Introducing Nunchaku 4-bit inference in Diffusers", section
"Background: SVDQuant and Nunchaku"):
    y = Q4(x_hat) . Q4(R) + (x_hat L1) L2 + b,  x_hat = bf16(x / lambda),
    R = diag(lambda) W - L1 L2,
with svdq_w4a4 NVFP4 (group 16) or INT4 (group 64) and awq_w4a16 INT4
(group 64) (Diffusers "Nunchaku Lite" page, table "Supported quantization
types").
"""

from __future__ import annotations

import ctypes as C
import enum
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

__all__ = [
    "NVFP4", "INT4", "Status", "SvdqError", "PackedWeight", "QuantAct", "AwqWeight",
    "library_path", "load", "scale_bytes", "pack_weight", "quantize_act", "w4a4_linear",
    "w4a4_linear_qkv", "qkv_norm_rope", "RopeTable", "pack_rope", "svdq_linear", "awq_pack_weight", "awq_w4a16_linear",
    "Fp8Act", "Fp8Weight", "fp8_quantize_act", "fp8_norm_quantize", "fp8_pack_weight", "fp8_linear",
    "RopeFreqs", "rope_freqs", "rope_tables", "rope_apply", "device_error", "set_wait_limit_ns",
    "probe_convert", "probe_wait_timeout", "probe_mma_peak", "probe_fp8_linear_plan", "probe_fp8_act_plan",
    "debug_force_arch",
]

NVFP4, INT4 = 0, 1
_OUT = {"bf16": 0, "f32": 1, "i32_groups": 2, "bf16_gelu": 3}
_ROPE_LAYOUT = {"interleaved": 0, "half": 1}
_HERE = os.path.dirname(os.path.abspath(__file__))


class Status(enum.IntEnum):
    OK = 0
    INVALID_ARG = 1
    SHAPE = 2
    ALIGN = 3
    UNSUPPORTED_ARCH = 4
    CUDA = 5
    TIMEOUT = 6


class SvdqError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = Status(status)


_lib = None


def library_path() -> str:
    return os.path.join(_HERE, "libsvdq.so")


# name -> (restype, argtypes)
_P, _I, _F, _U64, _I64 = C.c_void_p, C.c_int, C.c_float, C.c_ulonglong, C.c_longlong
SIGNATURES = {
    "svdq_status_str": (C.c_char_p, [_I]),
    "svdq_scale_bytes": (C.c_size_t, [_I, _I, _I]),
    "svdq_lr_up_elems": (C.c_size_t, [_I, _I, _I]),
    "svdq_pack_weight": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _F, _P, _P, _P, _P, _P, _P]),
    "svdq_quantize_act": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "svdq_w4a4_linear": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P]),
    "svdq_rope_packed_bytes": (C.c_size_t, [_I]),
    "svdq_rope_pack": (_I, [_I, _P, _P, _P, _P]),
    "svdq_w4a4_linear_qkv": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P]),
    "svdq_qkv_norm_rope": (_I, [_I, _I, _P, _P, _F, _P, _P, _P, _P]),
    "awq_pack_weight": (_I, [_I, _I, _P, _P, _P, _P, _P]),
    "awq_w4a16_linear": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "svdq_fp8_quantize_act": (_I, [_I, _I, _P, _I64, _P, _P, _P]),
    "svdq_fp8_norm_quantize": (_I, [_I, _I, _P, _I64, _P, _I64, _P, _F, _P, _I64, _P, _P, _P]),
    "svdq_fp8_pack_weight": (_I, [_I, _I, _P, _P, _P, _P]),
    "svdq_fp8_linear": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P]),
    "svdq_rope_tables": (_I, [_I, _I, _I, _P, _P, _P, _F, _P, _P, _P]),
    "svdq_rope_apply": (_I, [_I, _I, _I, _I, _I, _I, _P, _P, _P, _F, _P, _I64, _P, _I64, _P]),
    "svdq_device_error": (_I, [_P]),
    "svdq_set_wait_limit_ns": (None, [_U64]),
    "svdq_probe_convert": (_I, [_P, _I64, _P, _P, _P, _P]),
    "svdq_probe_wait_timeout": (_I, [_U64, _P]),
    "svdq_probe_fp8_linear_plan": (_I, [_I, _I, _I, _I, _P]),
    "svdq_probe_fp8_act_plan": (_I, [_I, _I, _I, _I, _I, _P]),
    "svdq_debug_force_arch": (None, [_I, _I]),
    "svdq_probe_mma_peak": (_I, [_I, _I, _P]),
}


def load():
    """Load ``libsvdq.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m bit_w4a4_quantized_nvfp4_b200.build` "
                "(nvcc, sm_100a); this package has no fallback implementation")
        L = C.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise SvdqError(fn, status, load().svdq_status_str(status).decode())


def _ptr(t: Optional[torch.Tensor], dev: Optional[int] = None):
    """Device address of a contiguous CUDA tensor on the current device
    (``dev``, when the caller has already read it)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    cur = torch.cuda.current_device() if dev is None else dev
    if t.get_device() != cur:
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{cur}")
    return t.data_ptr()


def _ptrs(*ts):
    """_ptr of several tensors, reading the current device once."""
    dev = None
    out = []
    for t in ts:
        if t is not None and dev is None:
            if not t.is_cuda:
                raise ValueError("expected a CUDA tensor")
            dev = torch.cuda.current_device()
        out.append(_ptr(t, dev))
    return out


def _need(cond: bool, what, *args) -> None:
    """Argument check of the binding: the C ABI receives bare pointers and
    cannot see sizes, so every shape and dtype is checked here, before any
    pointer reaches the library (a wrong size would otherwise become a read
    or write past an allocation). The message is formatted only on failure."""
    if not cond:
        raise ValueError(what.format(*args) if args else what)


def _is(t: Optional[torch.Tensor], dtype, shape, name: str) -> None:
    if t is None:
        raise ValueError(f"{name}: missing")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _at_least(t: torch.Tensor, dtype, nbytes: int, name: str) -> None:
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, need {nbytes}")


# the current stream's handle without building a Stream object (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None, dev: Optional[int] = None):
    """Handle of ``stream``, or of the current one on the current device
    (``dev``, when the caller has already read it)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if dev is None else dev)
    return torch.cuda.current_stream().cuda_stream


def _prec(p) -> int:
    if isinstance(p, str):
        return {"nvfp4": NVFP4, "int4": INT4}[p]
    return int(p)


def scale_bytes(prec, rows: int, K: int) -> int:
    return int(load().svdq_scale_bytes(_prec(prec), rows, K))


@dataclass
class PackedWeight:
    prec: int
    K: int
    N: int
    r: int
    codes: torch.Tensor          # uint8 [N, K/2]
    scales: torch.Tensor         # uint8 (tiled e4m3 bytes or bf16 pairs)
    tensor_scale: torch.Tensor   # float32 [2] = {s_tw, s_tx}
    inv_lambda: torch.Tensor     # float32 [K]
    lr_up: Optional[torch.Tensor]  # bf16 [N, 2r] (NVFP4) or [N, r] (INT4)
    act_tensor_scale: float


@dataclass
class QuantAct:
    prec: int
    M: int
    K: int
    r: int
    codes: torch.Tensor    # uint8 [M, K/2]
    scales: torch.Tensor   # uint8 bytes
    P: Optional[torch.Tensor]  # bf16 [M, r]


def _check_packed(pw: PackedWeight) -> None:
    """The buffers of a packed weight have the sizes its (prec, K, N, r) imply."""
    _need(pw.prec in (NVFP4, INT4), "precision {!r}", pw.prec)
    _is(pw.codes, torch.uint8, (pw.N, pw.K // 2), "pw.codes")
    _at_least(pw.scales, torch.uint8, scale_bytes(pw.prec, pw.N, pw.K), "pw.scales")
    _is(pw.tensor_scale, torch.float32, (2,), "pw.tensor_scale")
    _is(pw.inv_lambda, torch.float32, (pw.K,), "pw.inv_lambda")
    if pw.r:
        _is(pw.lr_up, torch.bfloat16, (pw.N, 2 * pw.r if pw.prec == NVFP4 else pw.r), "pw.lr_up")


def pack_weight(prec, W: torch.Tensor, lam: torch.Tensor, L1: Optional[torch.Tensor],
                L2: Optional[torch.Tensor], act_tensor_scale: float = 1.0, stream=None) -> PackedWeight:
    """svdq_pack_weight: W fp32 [K, N], lam fp32 [K], L1 bf16 [K, r], L2 bf16 [r, N]."""
    p = _prec(prec)
    _need(p in (NVFP4, INT4), "precision {!r}", prec)
    _need(W.dim() == 2 and W.dtype == torch.float32, "W: expected float32 [K, N]")
    K, N = W.shape
    r = 0 if L1 is None else L1.shape[1]
    _is(lam, torch.float32, (K,), "lambda")
    if r:
        _is(L1, torch.bfloat16, (K, r), "L1")
        _is(L2, torch.bfloat16, (r, N), "L2")
    else:
        _need(L2 is None or L2.numel() == 0, "L2 given without L1")
    dev = W.device
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty(max(scale_bytes(p, N, K), 16), dtype=torch.uint8, device=dev)
    ts = torch.empty(4, dtype=torch.float32, device=dev)[:2]
    inv = torch.empty(K, dtype=torch.float32, device=dev)
    rr = (2 * r if p == NVFP4 else r)
    lr_up = torch.empty((N, rr), dtype=torch.bfloat16, device=dev) if r else None
    _check("svdq_pack_weight", load().svdq_pack_weight(
        p, K, N, r, _ptr(W), _ptr(lam), _ptr(L1), _ptr(L2), float(act_tensor_scale), _ptr(codes),
        _ptr(scales), _ptr(ts), _ptr(inv), _ptr(lr_up), _stream(stream)))
    return PackedWeight(p, K, N, r, codes, scales, ts, inv, lr_up, float(act_tensor_scale))


def quantize_act(x: torch.Tensor, pw: PackedWeight, L1: Optional[torch.Tensor], stream=None,
                 out: Optional[QuantAct] = None) -> QuantAct:
    """svdq_quantize_act: x bf16 [M, K] -> codes, scales, P. The activation
    tensor scale is the one packed into ``pw.tensor_scale`` (read on the device)."""
    _need(x.dim() == 2 and x.dtype == torch.bfloat16, "x: expected bfloat16 [M, K]")
    M, K = x.shape
    _check_packed(pw)
    p, r = pw.prec, pw.r
    _need(K == pw.K, "x has K = {}, the packed weight K = {}", K, pw.K)
    if r:
        _is(L1, torch.bfloat16, (K, r), "L1")
    dev = x.device
    if out is None:
        out = QuantAct(p, M, K, r, torch.empty((M, K // 2), dtype=torch.uint8, device=dev),
                       torch.empty(max(scale_bytes(p, M, K), 16), dtype=torch.uint8, device=dev),
                       torch.empty((M, r), dtype=torch.bfloat16, device=dev) if r else None)
    else:
        _need(out.prec == p and out.M == M and out.K == K and out.r == r,
              "out: QuantAct of another shape or precision")
        _is(out.codes, torch.uint8, (M, K // 2), "out.codes")
        _at_least(out.scales, torch.uint8, scale_bytes(p, M, K), "out.scales")
        if r:
            _is(out.P, torch.bfloat16, (M, r), "out.P")
    px, pil, pts, pl1, pc, psc, pp = _ptrs(x, pw.inv_lambda, pw.tensor_scale, L1, out.codes, out.scales, out.P)
    _check("svdq_quantize_act", load().svdq_quantize_act(p, M, K, r, px, pil, pts, pl1, pc, psc, pp, _stream(stream)))
    return out


def w4a4_linear(qa: QuantAct, pw: PackedWeight, bias: Optional[torch.Tensor] = None,
                out_dtype: str = "bf16", stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """svdq_w4a4_linear: the 4-bit GEMM with the low-rank up-projection and bias fused."""
    M, K, N = qa.M, qa.K, pw.N
    _check_packed(pw)
    _need(qa.prec == pw.prec and qa.K == pw.K and qa.r == pw.r,
          "activations (prec {}, K {}, r {}) do not match the weight (prec {}, K {}, r {})",
          qa.prec, qa.K, qa.r, pw.prec, pw.K, pw.r)
    _is(qa.codes, torch.uint8, (M, K // 2), "qa.codes")
    _at_least(qa.scales, torch.uint8, scale_bytes(qa.prec, M, K), "qa.scales")
    if qa.r:
        _is(qa.P, torch.bfloat16, (M, qa.r), "qa.P")
    if bias is not None:
        _is(bias, torch.bfloat16, (N,), "bias")
    _need(out_dtype in _OUT, "out_dtype {!r}", out_dtype)
    want = {"bf16": (torch.bfloat16, (M, N)), "f32": (torch.float32, (M, N)),
            "i32_groups": (torch.int32, (M, N, K // 64)), "bf16_gelu": (torch.bfloat16, (M, N))}[out_dtype]
    if out is not None:
        _is(out, want[0], want[1], "out")
    if out is None:
        if out_dtype in ("bf16", "bf16_gelu"):
            out = torch.empty((M, N), dtype=torch.bfloat16, device=qa.codes.device)
        elif out_dtype == "f32":
            out = torch.empty((M, N), dtype=torch.float32, device=qa.codes.device)
        else:
            out = torch.empty((M, N, K // 64), dtype=torch.int32, device=qa.codes.device)
    ptrs = _ptrs(qa.codes, qa.scales, qa.P, pw.codes, pw.scales, pw.tensor_scale, pw.lr_up, bias, out)
    _check("svdq_w4a4_linear", load().svdq_w4a4_linear(pw.prec, M, K, N, pw.r, *ptrs, _OUT[out_dtype],
                                                       _stream(stream)))
    return out


@dataclass
class RopeTable:
    """The rotary cos/sin tables of M rows in svdq_rope_pack's layout (fp32,
    svdq_rope_packed_bytes(M) bytes)."""
    M: int
    data: torch.Tensor


def pack_rope(cos: torch.Tensor, sin: torch.Tensor, stream=None) -> RopeTable:
    """svdq_rope_pack: cos, sin fp32 [M, 64] -> the packed table the fused QKV
    epilogue reads (once per set of positions; every layer can share it)."""
    _need(cos.dim() == 2, "cos: expected [M, 64]")
    M = cos.shape[0]
    _is(cos, torch.float32, (M, 64), "cos")
    _is(sin, torch.float32, (M, 64), "sin")
    data = torch.empty(load().svdq_rope_packed_bytes(M) // 4, dtype=torch.float32, device=cos.device)
    pc, ps, pr = _ptrs(cos, sin, data)
    _check("svdq_rope_pack", load().svdq_rope_pack(M, pc, ps, pr, _stream(stream)))
    return RopeTable(M, data)


def w4a4_linear_qkv(qa: QuantAct, pw: PackedWeight, heads: int, norm_q: torch.Tensor, norm_k: torch.Tensor,
                    eps: float, rope: RopeTable, bias: Optional[torch.Tensor] = None,
                    stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """svdq_w4a4_linear_qkv: the NVFP4 layer as a grouped Q/K/V projection (N =
    3 * heads * 128) with per-head RMSNorm of Q and K and the rotary embedding
    in the GEMM's epilogue. rope: pack_rope of the M rows' cos/sin [M, 64]."""
    M, K, N = qa.M, qa.K, pw.N
    _check_packed(pw)
    _need(pw.prec == NVFP4 and qa.prec == NVFP4, "the fused QKV epilogue is NVFP4 only")
    _need(qa.K == pw.K and qa.r == pw.r, "activations (K {}, r {}) do not match the weight (K {}, r {})",
          qa.K, qa.r, pw.K, pw.r)
    _need(heads > 0 and N == 3 * heads * 128, "N = {} is not 3 * heads * 128 with heads = {}", N, heads)
    _is(qa.codes, torch.uint8, (M, K // 2), "qa.codes")
    _at_least(qa.scales, torch.uint8, scale_bytes(qa.prec, M, K), "qa.scales")
    if qa.r:
        _is(qa.P, torch.bfloat16, (M, qa.r), "qa.P")
    _is(norm_q, torch.bfloat16, (128,), "norm_q")
    _is(norm_k, torch.bfloat16, (128,), "norm_k")
    _need(isinstance(rope, RopeTable) and rope.M == M, "rope: expected pack_rope of the layer's {} rows", M)
    _is(rope.data, torch.float32, (load().svdq_rope_packed_bytes(M) // 4,), "rope.data")
    if bias is not None:
        _is(bias, torch.bfloat16, (N,), "bias")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=qa.codes.device)
    else:
        _is(out, torch.bfloat16, (M, N), "out")
    ptrs = _ptrs(qa.codes, qa.scales, qa.P, pw.codes, pw.scales, pw.tensor_scale, pw.lr_up, bias, norm_q, norm_k)
    pr, po = _ptrs(rope.data, out)
    _check("svdq_w4a4_linear_qkv", load().svdq_w4a4_linear_qkv(M, K, heads, pw.r, *ptrs, float(eps), pr, po,
                                                               _stream(stream)))
    return out


def qkv_norm_rope(y: torch.Tensor, heads: int, norm_q: torch.Tensor, norm_k: torch.Tensor, eps: float,
                  cos: torch.Tensor, sin: torch.Tensor, stream=None) -> torch.Tensor:
    """svdq_qkv_norm_rope: per-head RMSNorm + rotary embedding of the Q and K
    sections of a bf16 grouped-QKV output y [M, 3 * heads * 128], in place."""
    _need(y.dim() == 2 and y.dtype == torch.bfloat16, "y: expected bfloat16 [M, N]")
    M, N = y.shape
    _need(heads > 0 and N == 3 * heads * 128, "N = {} is not 3 * heads * 128 with heads = {}", N, heads)
    _is(norm_q, torch.bfloat16, (128,), "norm_q")
    _is(norm_k, torch.bfloat16, (128,), "norm_k")
    _is(cos, torch.float32, (M, 64), "cos")
    _is(sin, torch.float32, (M, 64), "sin")
    pq, pk, pc, ps, py = _ptrs(norm_q, norm_k, cos, sin, y)
    _check("svdq_qkv_norm_rope", load().svdq_qkv_norm_rope(M, heads, pq, pk, float(eps), pc, ps, py,
                                                           _stream(stream)))
    return y


def svdq_linear(x: torch.Tensor, pw: PackedWeight, L1: Optional[torch.Tensor],
                bias: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The whole layer: quantize_act then w4a4_linear (two launches)."""
    return w4a4_linear(quantize_act(x, pw, L1, stream), pw, bias, stream=stream)


@dataclass
class AwqWeight:
    K: int
    N: int
    q: torch.Tensor       # uint8 [N, K/2]
    scales: torch.Tensor  # bf16 [N, K/64]
    zeros: torch.Tensor   # bf16 [N, K/64]


def awq_pack_weight(W: torch.Tensor, stream=None, out: Optional[AwqWeight] = None) -> AwqWeight:
    """awq_pack_weight: W fp32 [K, N] -> q, scales, zeros (into ``out``'s
    buffers when given)."""
    _need(W.dim() == 2 and W.dtype == torch.float32, "W: expected float32 [K, N]")
    K, N = W.shape
    dev = W.device
    if out is None:
        out = AwqWeight(K, N, torch.empty((N, K // 2), dtype=torch.uint8, device=dev),
                        torch.empty((N, K // 64), dtype=torch.bfloat16, device=dev),
                        torch.empty((N, K // 64), dtype=torch.bfloat16, device=dev))
    else:
        _need(out.K == K and out.N == N, "out: AwqWeight of K {}, N {}", out.K, out.N)
        _is(out.q, torch.uint8, (N, K // 2), "out.q")
        _is(out.scales, torch.bfloat16, (N, K // 64), "out.scales")
        _is(out.zeros, torch.bfloat16, (N, K // 64), "out.zeros")
    _check("awq_pack_weight", load().awq_pack_weight(K, N, _ptr(W), _ptr(out.q), _ptr(out.scales),
                                                     _ptr(out.zeros), _stream(stream)))
    return out


def awq_w4a16_linear(x: torch.Tensor, w: AwqWeight, bias: Optional[torch.Tensor] = None, stream=None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _need(x.dim() == 2 and x.dtype == torch.bfloat16, "x: expected bfloat16 [M, K]")
    M, K = x.shape
    _need(K == w.K, "x has K = {}, the packed weight K = {}", K, w.K)
    _is(w.q, torch.uint8, (w.N, w.K // 2), "w.q")
    _is(w.scales, torch.bfloat16, (w.N, w.K // 64), "w.scales")
    _is(w.zeros, torch.bfloat16, (w.N, w.K // 64), "w.zeros")
    if bias is not None:
        _is(bias, torch.bfloat16, (w.N,), "bias")
    if out is not None:
        _is(out, torch.bfloat16, (M, w.N), "out")
    if out is None:
        out = torch.empty((M, w.N), dtype=torch.bfloat16, device=x.device)
    _check("awq_w4a16_linear", load().awq_w4a16_linear(
        M, K, w.N, _ptr(x), _ptr(w.q), _ptr(w.scales), _ptr(w.zeros), _ptr(bias), _ptr(out),
        _stream(stream)))
    return out


# ------------------------------------------------------------------ the 8-bit linear layer
@dataclass
class Fp8Act:
    """bf16 activations in 8 bits: E4M3 codes and one fp32 scale per 128 columns of a row."""
    M: int
    K: int
    codes: torch.Tensor   # float8_e4m3fn [M, K]
    scales: torch.Tensor  # float32 [ceil(K/128), M]


@dataclass
class Fp8Weight:
    """A weight in 8 bits: E4M3 codes and one fp32 scale per 128 x 128 block."""
    K: int
    N: int
    codes: torch.Tensor   # float8_e4m3fn [N, K]
    scales: torch.Tensor  # float32 [ceil(N/128), ceil(K/128)]


# (bound once: these calls are as short as the host makes them)
_F8, _BF16, _F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
_device, _empty_strided = torch.cuda.current_device, torch.empty_strided


def _blocks(n: int) -> int:
    return (n + 127) // 128


# Sizes go to the library as C ints, which ctypes would wrap.
_MOST = 0x7FFFFFFF


def _too_large(*sizes: int) -> None:
    raise ValueError(f"size {max(sizes)}: 2^31 - 1 is the largest")


def _rows(t: torch.Tensor, name: str):
    """(M, K, row stride in elements) of a bf16 [M, K] tensor whose rows may
    be a column range of a wider tensor: unit column stride, and rows that
    follow one another without overlap (a stride in a dimension of size one
    says nothing and is not looked at)."""
    if t.dtype is not _BF16 or t.dim() != 2:
        raise ValueError(f"{name}: expected bfloat16 [M, K]")
    M, K = t.shape
    if M > _MOST or K > _MOST:
        _too_large(M, K)
    s0, s1 = t.stride()
    if s1 != 1 and K > 1:
        raise ValueError(f"{name}: expected unit stride along the columns")
    if M <= 1:
        return M, K, (K + 7) // 8 * 8
    if s0 < K:
        raise ValueError(f"{name}: row stride {s0} is less than the row's {K} columns")
    return M, K, s0


def _rows_as(t: torch.Tensor, name: str, M: int, K: int) -> int:
    """Row stride of such a tensor of M rows of K columns."""
    m, k, ld = _rows(t, name)
    if m != M or k != K:
        raise ValueError(f"{name}: shape {(m, k)}, expected {(M, K)}")
    return ld


def _addr(t: torch.Tensor, dev: int, name: str) -> int:
    """Device address of a CUDA tensor of any strides on device ``dev``."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor")
        raise ValueError(f"{name}: tensor on {t.device}, but the current device is cuda:{dev}")
    return t.data_ptr()


def _flat(t: Optional[torch.Tensor], dev: int, name: str):
    """Device address of a contiguous CUDA tensor on device ``dev`` (None: none)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return _addr(t, dev, name)


def _current(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return _device()


def _new(rows: int, cols: int, dtype, device, stream) -> torch.Tensor:
    """A contiguous output [rows, cols] of a call on ``stream``, allocated for
    the stream that writes it (empty_strided takes two thirds of empty's time)."""
    if stream is None:
        return _empty_strided((rows, cols), (cols or 1, 1), dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return _empty_strided((rows, cols), (cols or 1, 1), dtype=dtype, device=device)


def _fp8_act_out(out: Optional[Fp8Act], M: int, K: int, x: torch.Tensor, stream, dev: int):
    """(the Fp8Act of a call, the addresses of its codes and scales)"""
    G = (K + 127) // 128
    if out is None:
        device = x.device
        codes, scales = _new(M, K, _F8, device, stream), _new(G, M, _F32, device, stream)
        return Fp8Act(M, K, codes, scales), codes.data_ptr(), scales.data_ptr()
    if out.M != M or out.K != K:
        raise ValueError(f"out: Fp8Act of M {out.M}, K {out.K}")
    _is(out.codes, _F8, (M, K), "out.codes")
    _is(out.scales, _F32, (G, M), "out.scales")
    return out, _flat(out.codes, dev, "out.codes"), _flat(out.scales, dev, "out.scales")


def fp8_quantize_act(x: torch.Tensor, stream=None, out: Optional[Fp8Act] = None) -> Fp8Act:
    """svdq_fp8_quantize_act: x bf16 [M, K] (rows may be strided) -> codes, scales."""
    M, K, ldx = _rows(x, "x")
    dev = _current(x)
    px = _addr(x, dev, "x")
    out, pc, ps = _fp8_act_out(out, M, K, x, stream, dev)
    _check("svdq_fp8_quantize_act", load().svdq_fp8_quantize_act(M, K, px, ldx, pc, ps, _stream(stream, dev)))
    return out


def fp8_norm_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                      stream=None, out: Optional[Fp8Act] = None, residual_out: Optional[torch.Tensor] = None):
    """svdq_fp8_norm_quantize: r = bf16(x + residual), then the 8-bit form of
    RMSNorm(r) * weight. Returns (Fp8Act, r); r is None without a residual.
    x, residual and residual_out bf16 [M, K], rows may be strided;
    residual_out may be x or residual (in place)."""
    M, K, ldx = _rows(x, "x")
    _is(weight, _BF16, (K,), "weight")
    dev = _current(x)
    px, pw = _addr(x, dev, "x"), _flat(weight, dev, "weight")
    pr = po = None
    ldr = ldo = 0
    if residual is not None:
        ldr = _rows_as(residual, "residual", M, K)
        pr = _addr(residual, dev, "residual")
        if residual_out is None:
            residual_out = _new(M, K, _BF16, x.device, stream)
            ldo = (K + 7) // 8 * 8
            po = residual_out.data_ptr()
        else:
            ldo = _rows_as(residual_out, "residual_out", M, K)
            po = _addr(residual_out, dev, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out given without residual")
    out, pc, ps = _fp8_act_out(out, M, K, x, stream, dev)
    _check("svdq_fp8_norm_quantize", load().svdq_fp8_norm_quantize(
        M, K, px, ldx, pr, ldr, pw, float(eps), po, ldo, pc, ps, _stream(stream, dev)))
    return out, residual_out


def fp8_pack_weight(W: torch.Tensor, stream=None, out: Optional[Fp8Weight] = None) -> Fp8Weight:
    """svdq_fp8_pack_weight: W fp32 [K, N] -> codes, scales (into ``out``'s buffers when given)."""
    _need(W.dim() == 2 and W.dtype == torch.float32, "W: expected float32 [K, N]")
    K, N = W.shape
    if K > _MOST or N > _MOST:
        _too_large(K, N)
    dev = _current(W)
    if out is None:
        out = Fp8Weight(K, N, _new(N, K, _F8, W.device, stream),
                        _new(_blocks(N), _blocks(K), torch.float32, W.device, stream))
    else:
        _need(out.K == K and out.N == N, "out: Fp8Weight of K {}, N {}", out.K, out.N)
        _is(out.codes, _F8, (N, K), "out.codes")
        _is(out.scales, torch.float32, (_blocks(N), _blocks(K)), "out.scales")
    _check("svdq_fp8_pack_weight", load().svdq_fp8_pack_weight(
        K, N, _flat(W, dev, "W"), _flat(out.codes, dev, "out.codes"), _flat(out.scales, dev, "out.scales"),
        _stream(stream, dev)))
    return out


def fp8_linear(qa: Fp8Act, w: Fp8Weight, bias: Optional[torch.Tensor] = None, out_dtype: str = "bf16", stream=None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """svdq_fp8_linear: y [M, N] = the product of the 8-bit operands, + bias. out_dtype "bf16" or "f32"."""
    M, K, N = qa.M, qa.K, w.N
    if K != w.K:
        raise ValueError(f"activations have K = {K}, the packed weight K = {w.K}")
    _need(out_dtype == "bf16" or out_dtype == "f32", "out_dtype {!r}", out_dtype)
    if M > _MOST or K > _MOST or N > _MOST:
        _too_large(M, K, N)
    G = (K + 127) // 128
    xc, xs, wc, ws = qa.codes, qa.scales, w.codes, w.scales
    _is(xc, _F8, (M, K), "qa.codes")
    _is(xs, _F32, (G, M), "qa.scales")
    _is(wc, _F8, (N, K), "w.codes")
    _is(ws, _F32, ((N + 127) // 128, G), "w.scales")
    if bias is not None:
        _is(bias, _BF16, (N,), "bias")
    want = _BF16 if out_dtype == "bf16" else _F32
    dev = _current(xc)
    pxc, pxs = _flat(xc, dev, "qa.codes"), _flat(xs, dev, "qa.scales")
    pwc, pws, pb = _flat(wc, dev, "w.codes"), _flat(ws, dev, "w.scales"), _flat(bias, dev, "bias")
    if out is None:
        out = _new(M, N, want, xc.device, stream)
        po = out.data_ptr()
    else:
        _is(out, want, (M, N), "out")
        po = _flat(out, dev, "out")
    _check("svdq_fp8_linear", load().svdq_fp8_linear(
        M, K, N, pxc, pxs, pwc, pws, pb, po, _OUT[out_dtype], _stream(stream, dev)))
    return out


# ------------------------------------------------------------------ rotary positions
@dataclass
class RopeFreqs:
    """How rotary pairs turn: freq float64 [pairs], radians per position; the
    factor on cos and sin; axis int32 [pairs], the position axis of each pair
    (None: all pairs follow axis 0). Made once per model (rope_freqs)."""
    freq: torch.Tensor
    factor: float = 1.0
    axis: Optional[torch.Tensor] = None


def rope_freqs(rot_dim, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
               original_len: int = 0, device="cuda") -> RopeFreqs:
    """The frequencies of heads whose first ``rot_dim`` columns turn: base **
    (-2 i / rot_dim) for pair i, in 64 bits. rot_dim: an even number, or one
    per position axis (their pairs follow one another).

    scaling for contexts ``factor`` times longer than the trained one:
      None      none
      "linear"  every frequency divided by the factor
      "ntk"     a larger base, with which the slowest pair slows by the factor
                and the fastest keeps its frequency
      "yarn"    pairs that turn less than once within original_len slow by the
                factor, those that turn more than 32 times stay, a linear ramp
                over the pair index between them; cos and sin times
                0.1 ln(factor) + 1
    """
    dims = [int(rot_dim)] if isinstance(rot_dim, int) else [int(d) for d in rot_dim]
    _need(1 <= len(dims) <= 8 and all(d >= 2 and d % 2 == 0 for d in dims), "rot_dim {!r}: even numbers expected",
          rot_dim)
    _need(scaling in (None, "linear", "ntk", "yarn"), "scaling {!r}", scaling)
    _need(base > 1.0 and factor >= 1.0 and math.isfinite(base) and math.isfinite(factor), "base {}, factor {}",
          base, factor)
    _need(scaling != "yarn" or original_len > 0, "yarn needs original_len")
    parts, mult = [], 1.0
    for d in dims:
        i = torch.arange(d // 2, dtype=torch.float64)
        b = base * factor ** (d / (d - 2)) if scaling == "ntk" and d > 2 else base
        f = b ** (-2.0 * i / d)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            # the (real-valued) pair index at which a pair turns `turns` times within original_len
            def pair(turns):
                return d * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
            lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), d - 1)
            # (no ramp where not even the first pair turns once, or all turn 32 times)
            slow = ((i - lo) / (hi - lo)).clamp(0.0, 1.0) if hi > lo else (i >= hi).to(torch.float64)
            f = f / factor * slow + f * (1.0 - slow)
            mult = 0.1 * math.log(factor) + 1.0
        parts.append(f)
    axis = None
    if len(dims) > 1:
        axis = torch.repeat_interleave(torch.arange(len(dims), dtype=torch.int32), torch.tensor(dims) // 2).to(device)
    return RopeFreqs(torch.cat(parts).to(device), mult, axis)


def _rope_inputs(positions: torch.Tensor, freqs: RopeFreqs):
    """(current device, M, axes, pairs, and the addresses of pos, freq, axis) of a rotary call, checked."""
    shape = positions.shape
    if positions.dtype is not torch.int64 or len(shape) not in (1, 2):
        raise ValueError("positions: expected int64 [M] or [M, axes]")
    M, axes = shape if len(shape) == 2 else (shape[0], 1)
    f, axis = freqs.freq, freqs.axis
    if f.dtype is not torch.float64 or f.dim() != 1:
        raise ValueError("freqs.freq: expected float64 [pairs]")
    pairs = f.shape[0]
    if M > _MOST or axes > _MOST or pairs > _MOST:
        _too_large(M, axes, pairs)
    if axis is not None:
        _is(axis, torch.int32, (pairs,), "freqs.axis")
    dev = _current(positions)
    return (dev, M, axes, pairs, _flat(positions, dev, "positions"), _flat(f, dev, "freqs.freq"),
            _flat(axis, dev, "freqs.axis"))


def rope_tables(positions: torch.Tensor, freqs: RopeFreqs, stream=None):
    """svdq_rope_tables: (cos, sin) fp32 [M, pairs] at positions int64 [M] or
    [M, axes], the tables that pack_rope (pairs = 64) and qkv_norm_rope take."""
    dev, M, axes, pairs, pp, pf, pa = _rope_inputs(positions, freqs)
    device = positions.device
    cos, sin = _new(M, pairs, _F32, device, stream), _new(M, pairs, _F32, device, stream)
    _check("svdq_rope_tables", load().svdq_rope_tables(M, axes, pairs, pp, pf, pa, float(freqs.factor),
                                                       cos.data_ptr(), sin.data_ptr(), _stream(stream, dev)))
    return cos, sin


def rope_apply(x: torch.Tensor, heads: int, head_dim: int, positions: torch.Tensor, freqs: RopeFreqs,
               layout: str = "interleaved", stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """svdq_rope_apply: rotates the first 2 * pairs columns of each of the
    first ``heads`` heads of x bf16 [M, >= heads * head_dim] (rows may be
    strided: x may be a whole Q/K/V projection, whose Q and K heads come
    first). In place unless ``out`` [M, heads * head_dim] is given; returns
    what was written to."""
    _need(layout in _ROPE_LAYOUT, "layout {!r}", layout)
    rows, cols, ldx = _rows(x, "x")
    width = heads * head_dim
    _need(heads >= 1 and head_dim >= 1 and cols >= width, "x has {} columns, {} heads of {} need {}",
          cols, heads, head_dim, width)
    dev, M, axes, pairs, pp, pf, pa = _rope_inputs(positions, freqs)
    px = _addr(x, dev, "x")
    _need(M == rows, "positions: {} rows, x has {}", M, rows)
    if out is None:
        out, py, ldy = x, px, ldx
    else:
        ldy = _rows_as(out, "out", M, width)
        py = _addr(out, dev, "out")
    _check("svdq_rope_apply", load().svdq_rope_apply(
        M, heads, head_dim, pairs, _ROPE_LAYOUT[layout], axes, pp, pf, pa, float(freqs.factor), px, ldx, py, ldy,
        _stream(stream, dev)))
    return out


def device_error() -> int:
    """Reads and clears the device error word; raises SvdqError if it was set."""
    bits = C.c_uint(0)
    st = load().svdq_device_error(C.byref(bits))
    if st not in (0, int(Status.TIMEOUT), int(Status.CUDA)):
        _check("svdq_device_error", st)
    if st:
        raise SvdqError("svdq_device_error", st, f"device error word = {bits.value:#x}")
    return bits.value


def set_wait_limit_ns(ns: int) -> None:
    load().svdq_set_wait_limit_ns(int(ns))


def probe_convert(x: torch.Tensor, e2m1: bool = True, e4m3: bool = True, bf16: bool = True, stream=None):
    n = x.numel()
    o1 = torch.empty(n, dtype=torch.uint8, device=x.device) if e2m1 else None
    o2 = torch.empty(n, dtype=torch.uint8, device=x.device) if e4m3 else None
    o3 = torch.empty(n, dtype=torch.int16, device=x.device) if bf16 else None
    _check("svdq_probe_convert", load().svdq_probe_convert(_ptr(x), n, _ptr(o1), _ptr(o2), _ptr(o3),
                                                           _stream(stream)))
    return o1, o2, o3


def probe_wait_timeout(limit_ns: int, stream=None) -> None:
    _check("svdq_probe_wait_timeout", load().svdq_probe_wait_timeout(int(limit_ns), _stream(stream)))


def probe_mma_peak(iters: int, mode: int = 0, stream=None) -> float:
    """Launches the tensor-core rate probe; returns the FLOPs it performs (the
    caller times it on its stream)."""
    _check("svdq_probe_mma_peak", load().svdq_probe_mma_peak(int(iters), int(mode), _stream(stream)))
    sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return float(sms // 2) * iters * 4 * 2.0 * 256 * 256 * 64


def probe_fp8_linear_plan(M: int, K: int, N: int, sms: int):
    """(tokens of a tile, parts of K) that svdq_fp8_linear takes for few rows, (256, long run) for many."""
    plan = (C.c_int * 2)()
    _check("svdq_probe_fp8_linear_plan", load().svdq_probe_fp8_linear_plan(M, K, N, sms, plan))
    return tuple(plan)


def probe_fp8_act_plan(M: int, K: int, norm: bool, residual: bool, sms: int):
    """(loads in flight, warps of a row) that the 8-bit activation pass takes."""
    plan = (C.c_int * 2)()
    _check("svdq_probe_fp8_act_plan", load().svdq_probe_fp8_act_plan(M, K, int(norm), int(residual), sms, plan))
    return tuple(plan)


def debug_force_arch(major: int, minor: int = 0) -> None:
    load().svdq_debug_force_arch(int(major), int(minor))
