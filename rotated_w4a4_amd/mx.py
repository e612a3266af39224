"""MXFP4 linear layers: binding of the library's mx calls.

    qw, sw = mx_pack_weight(t, w)             # offline, w [K, N] (or layout="nk")
    qa, sa = mx_quantize_act(t, x)            # x [M, K]; t None: no rotation
    y = mx_gemm(qa, sa, qw, sw)               # [M, N] bf16 (or fp32)

Codes are FP4 E2M1, uint8 [rows, K / 2] with the even channel in the low four bits; scales are exponents plus 127
(E8M0), uint8 [K / 128, rows, 4]: byte i of entry (g, r) belongs to channels 128 g + 32 i .. of row r.  mx_scale_rows
turns scales stored by rows ([rows, K / 32], as checkpoints hold them) into that order.

Marshalling and argument checks only, like the rest of the package; the prepare_ forms check once and launch again on
each call.  Every call works on the GPU of its tensors, whichever is current.
"""
from __future__ import annotations

import ctypes

import torch

from . import Transform, _on_gpu, _out, lib
from .kv import KVCall, _code, _launch

__all__ = ["mx_quantize_act", "prepare_mx_quantize_act", "mx_pack_weight", "mx_dequantize", "prepare_mx_dequantize",
           "mx_gemm", "prepare_mx_gemm", "mx_scale_rows"]

_p, _i64 = ctypes.c_void_p, ctypes.c_int64
lib.rw4_mx_quantize_act.argtypes = [_p, _p, ctypes.c_int, _i64, _i64, _i64, _p, _p, _p]
lib.rw4_mx_pack_weight.argtypes = [_p, _p, ctypes.c_int, _i64, _i64, _i64, _i64, _p, _p, _p]
lib.rw4_mx_dequantize.argtypes = [_p, _p, _i64, _i64, _p, ctypes.c_int, _i64, _p]
lib.rw4_mx_gemm.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _p, ctypes.c_int, _i64, _p]
for _name in ("rw4_mx_quantize_act", "rw4_mx_pack_weight", "rw4_mx_dequantize", "rw4_mx_gemm"):
    getattr(lib, _name).restype = ctypes.c_int

_U8, _BF16 = torch.uint8, torch.bfloat16


# The checks below look at each tensor once and in one expression: a small call is
# bound by the host (3.2 us of a call are the launch), and each attribute costs 0.05 to
# 0.1 us.  What fails is looked at again for its message.
def _outputs(rows, K, q, s, device, dev):
    """Codes and scales of `rows` rows: allocated, or checked."""
    if K <= 0 or K & 127:
        raise ValueError(f"K must be a positive multiple of 128, not {K}")
    if q is None:
        q = torch.empty(rows, K >> 1, dtype=_U8, device=device)
    else:
        _out("q", q, (rows, K >> 1), _U8, dev)
    if s is None:
        s = torch.empty(K >> 7, rows, 4, dtype=_U8, device=device)
    else:
        _out("s", s, (K >> 7, rows, 4), _U8, dev)
    return q, s


def _operand(name, q, s, dev):
    """(rows, K) of codes and scales that a call reads."""
    size = q.shape
    if len(size) == 2 and q.dtype is _U8 and s.dtype is _U8 and q.get_device() == dev and s.get_device() == dev \
            and q.is_contiguous() and s.is_contiguous():
        rows, half = size
        if half and not half & 63 and s.shape == (half >> 6, rows, 4):
            return rows, half << 1
        raise ValueError(f"{name}: K must be a multiple of 128 and scales [K / 128, rows, 4]")
    _on_gpu(f"{name} codes", q, dev)
    _on_gpu(f"{name} scales", s, dev)
    if len(size) != 2 or q.dtype is not _U8 or s.dtype is not _U8:
        raise ValueError(f"{name}: codes must be uint8 [rows, K / 2] and scales uint8")
    raise ValueError(f"{name}: codes and scales must be contiguous")


def _result(out, out_dtype, rows, cols, device, dev):
    """(output, its dtype's code, elements from one row to the next): allocated, or checked."""
    if out is None:
        dtype = _BF16 if out_dtype is None else out_dtype
        return torch.empty(rows, cols, dtype=dtype, device=device), _code(dtype), cols if cols > 0 else 1
    _on_gpu("out", out, dev)
    if out_dtype is not None and out.dtype is not out_dtype:
        raise TypeError(f"out must be {out_dtype}")
    if out.dim() != 2 or out.shape != (rows, cols) or (cols > 1 and out.stride(1) != 1):
        raise ValueError(f"out must be [{rows}, {cols}] with unit stride along its rows")
    return out, _code(out.dtype), _pitch(out)


def _pitch(t):
    """Elements from one row to the next (a single row may have any stride)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def mx_quantize_act(t: Transform | None, x, q=None, s=None):
    """Rotate (t: a block Hadamard of 128, 256 or 512 channels, None for no rotation) and quantize activations x [M, K]
    (bf16 / fp32, unit stride along K) to MXFP4; returns (q, s).

    Per 32 channels the scale is 2^(floor(log2 max) - 2); codes round to nearest, ties to even, and saturate at 6."""
    fn, args, dev, what, _, result = _quantize(t, x, q, s)
    _launch(fn, args, dev, what)
    return result


def prepare_mx_quantize_act(t: Transform | None, x, q=None, s=None) -> KVCall:
    """mx_quantize_act checked and marshalled once; calling the result runs it."""
    return KVCall(*_quantize(t, x, q, s))


def _quantize(t, x, q, s):
    dev = x.get_device()
    if dev < 0:
        _on_gpu("x", x)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride along K")
    M, K = x.shape
    handle = None
    if t is not None:
        if K != t.K:
            raise ValueError(f"x has {K} channels, the transform {t.K}")
        handle = t.handle
    q, s = _outputs(M, K, q, s, x.device, dev)
    args = (handle, x.data_ptr(), _code(x.dtype), M, K, x.stride(0) if M > 1 else K, q.data_ptr(), s.data_ptr())
    return lib.rw4_mx_quantize_act, args, dev, "rw4_mx_quantize_act", (t, x), (q, s)


def mx_pack_weight(t: Transform | None, w, layout: str = "kn", qw=None, sw=None):
    """Rotate and quantize weights to MXFP4 (offline). layout "kn": w is [K, N]; "nk": w is [N, K] (nn.Linear).

    Returns (qw uint8 [N, K / 2], sw uint8 [K / 128, N, 4])."""
    dev = _on_gpu("w", w)
    if w.dim() != 2 or layout not in ("kn", "nk"):
        raise ValueError('w must be 2-D, layout "kn" or "nk"')
    K, N = w.shape if layout == "kn" else w.shape[::-1]
    sk, sn = w.stride() if layout == "kn" else w.stride()[::-1]
    if t is not None and K != t.K:
        raise ValueError(f"w has {K} input channels, the transform {t.K}")
    qw, sw = _outputs(N, K, qw, sw, w.device, dev)
    if N == 1:
        sn = K * sk
    _launch(lib.rw4_mx_pack_weight, (None if t is None else t.handle, w.data_ptr(), _code(w.dtype), N, K, sk, sn,
                                     qw.data_ptr(), sw.data_ptr()), dev, "rw4_mx_pack_weight")
    return qw, sw


def mx_dequantize(q, s, out_dtype=None, out=None):
    """The values [rows, K] of codes and scales, exact in bf16 (default) and fp32; a scale of 255 gives NaN, what is 2^128
    or more (large codes with scales of 2^126 and 2^127) infinity."""
    fn, args, dev, what, _, result = _dequantize(q, s, out_dtype, out)
    _launch(fn, args, dev, what)
    return result


def prepare_mx_dequantize(q, s, out_dtype=None, out=None) -> KVCall:
    """mx_dequantize checked and marshalled once; calling the result runs it."""
    return KVCall(*_dequantize(q, s, out_dtype, out))


def _dequantize(q, s, out_dtype, out):
    dev = q.get_device()
    if dev < 0:
        _on_gpu("q", q)
    rows, K = _operand("q", q, s, dev)
    out, code, pitch = _result(out, out_dtype, rows, K, q.device, dev)
    args = (q.data_ptr(), s.data_ptr(), rows, K, out.data_ptr(), code, pitch)
    return lib.rw4_mx_dequantize, args, dev, "rw4_mx_dequantize", (q, s), out


def mx_gemm(qa, sa, qw, sw, out_dtype=None, out=None):
    """Y [M, N] (bf16 by default, or fp32) of MXFP4 activations and weights, summed in fp32."""
    fn, args, dev, what, _, result = _gemm(qa, sa, qw, sw, out_dtype, out)
    _launch(fn, args, dev, what)
    return result


def prepare_mx_gemm(qa, sa, qw, sw, out_dtype=None, out=None) -> KVCall:
    """mx_gemm checked and marshalled once; calling the result runs it."""
    return KVCall(*_gemm(qa, sa, qw, sw, out_dtype, out))


def _gemm(qa, sa, qw, sw, out_dtype, out):
    dev = qa.get_device()
    if dev < 0:
        _on_gpu("qa", qa)
    M, K = _operand("a", qa, sa, dev)
    N, kw = _operand("w", qw, sw, dev)
    if kw != K:
        raise ValueError(f"activations have {K} channels, weights {kw}")
    out, code, pitch = _result(out, out_dtype, M, N, qa.device, dev)
    args = (qa.data_ptr(), sa.data_ptr(), qw.data_ptr(), sw.data_ptr(), M, N, K, out.data_ptr(), code, pitch)
    return lib.rw4_mx_gemm, args, dev, "rw4_mx_gemm", (qa, sa, qw, sw), out


def mx_scale_rows(s):
    """Scales [rows, K / 32] stored by rows, as the calls take them: uint8 [K / 128, rows, 4]."""
    rows, blocks = s.shape
    if s.dtype is not _U8 or blocks % 4:
        raise ValueError("scales must be uint8 [rows, K / 32] with K a multiple of 128")
    return s.reshape(rows, blocks // 4, 4).transpose(0, 1).contiguous()
