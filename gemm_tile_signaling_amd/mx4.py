"""4-bit (MX) operands and their product (``include/fo_ops.h``).

``mx4_quantize``, ``mx4_dequantize`` and ``mx4_gemm`` wrap the C calls of the
same names: argument checks and marshalling only.  Codes are uint8
[rows, 16 * blocks] and scales uint8 [ceil(blocks / 8), rows, 8], where a row
of ``cols`` values has ceil(cols / 32) blocks (``mx4_shapes``).  Outputs that
are not given are allocated by torch on the stream the call runs on.

Tensors must be on the current device.  As with every enqueue call of the
library, a tensor made on another stream must be ready before the call's
stream reaches it, and must live until the call has run.
"""

from __future__ import annotations

import ctypes as C
from typing import Optional

from . import _DTYPES, _check, _stream, lib

__all__ = ["mx4_shapes", "mx4_quantize", "mx4_dequantize", "mx4_gemm"]

_OUT_TYPES = dict(_DTYPES, fp32=2)
_bound = None


def _ops():
    """libfo.so with the signatures of the operators set."""
    global _bound
    if _bound is None:
        L = lib()
        vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
        for name, args in {
            "fo_mx4_quantize": [vp, i64, i64, i64, i32, vp, vp, vp],
            "fo_mx4_dequantize": [vp, vp, i64, i64, i32, vp, vp],
            "fo_mx4_gemm": [vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, vp],
            "fo_moe_workspace_bytes": [vp, vp],
            "fo_moe_forward": [vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
        }.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = C.c_int
        _bound = L
    return _bound


def _dtype_name(t) -> Optional[str]:
    import torch
    return {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}.get(t)


def _tensor(x, name: str, shape, itemsize: int, device=None) -> int:
    """Address of a contiguous device tensor of this shape and element size."""
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.element_size() != itemsize:
        raise ValueError(f"{name}: element size {x.element_size()} != {itemsize}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _on(x, name, device)
    return x.data_ptr()


def _on(x, name: str, device):
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")


def _current(x, name: str):
    """The device of ``x``, which must be the current one (the launch goes there)."""
    import torch
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if x.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {x.device}, the current device is cuda:{torch.cuda.current_device()}")
    return x.device


def _new(stream, device, *shapes_and_types):
    """Fresh tensors that belong to the stream the call runs on."""
    import torch
    if stream is None:
        return [torch.empty(s, dtype=t, device=device) for s, t in shapes_and_types]
    if isinstance(stream, int):
        raise ValueError("with a stream given as an address the outputs must be given too")
    with torch.cuda.stream(stream):
        return [torch.empty(s, dtype=t, device=device) for s, t in shapes_and_types]


def mx4_shapes(rows: int, cols: int):
    """Shapes of the codes and the scales of ``rows`` rows of ``cols`` values."""
    nb = -(-cols // 32)
    return (rows, 16 * nb), (-(-nb // 8), rows, 8)


def mx4_quantize(x, codes=None, scales=None, dtype: Optional[str] = None, stream=None):
    """Rows of bf16/fp16 values to (codes, scales) (``fo_mx4_quantize``).

    ``x`` [rows, cols]: unit stride along a row, any row stride of at least
    ``cols``.  ``dtype`` ("bf16" or "fp16") names the type of a 16-bit integer
    tensor that holds the bits; a bfloat16 or float16 tensor names its own."""
    import torch
    name = _dtype_name(x.dtype) or dtype
    if name not in _DTYPES or (dtype is not None and dtype != name) or x.element_size() != 2:
        raise ValueError(f"x: expected bfloat16 or float16 values, got {x.dtype} and dtype={dtype!r}")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [rows, cols]")
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    if (cols > 1 and x.stride(1) != 1) or ld < cols:
        raise ValueError(f"x: strides {x.stride()}, expected unit stride along a row and rows that do not overlap")
    device = _current(x, "x")
    cs, ss = mx4_shapes(rows, cols)
    if codes is None or scales is None:
        new = _new(stream, device, (cs, torch.uint8), (ss, torch.uint8))
        codes, scales = new[0] if codes is None else codes, new[1] if scales is None else scales
    _check(_ops().fo_mx4_quantize(x.data_ptr(), rows, cols, ld, _DTYPES[name], _tensor(codes, "codes", cs, 1, device),
                                  _tensor(scales, "scales", ss, 1, device), _stream(stream)), "fo_mx4_quantize")
    return codes, scales


def mx4_dequantize(codes, scales, cols: int, dtype: str = "bf16", out=None, stream=None):
    """The values [rows, cols] that codes and scales stand for (``fo_mx4_dequantize``);
    ``dtype``: "bf16", "fp16" or "fp32"."""
    import torch
    if dtype not in _OUT_TYPES:
        raise ValueError(f"dtype: {dtype!r}, expected one of {sorted(_OUT_TYPES)}")
    if cols < 1:
        raise ValueError(f"cols: {cols}, expected at least 1")
    rows = codes.shape[0]
    cs, ss = mx4_shapes(rows, cols)
    device = _current(codes, "codes")
    if out is None:
        out, = _new(stream, device, ((rows, cols), {"bf16": torch.bfloat16, "fp16": torch.float16,
                                                    "fp32": torch.float32}[dtype]))
    _check(_ops().fo_mx4_dequantize(
        _tensor(codes, "codes", cs, 1, device), _tensor(scales, "scales", ss, 1, device), rows, cols,
        _OUT_TYPES[dtype], _tensor(out, "out", (rows, cols), 4 if dtype == "fp32" else 2, device), _stream(stream)),
        "fo_mx4_dequantize")
    return out


def mx4_gemm(a_codes, a_scales, b_codes, b_scales, dtype: str = "bf16", row_ends=None, out=None, stream=None):
    """out [M, N] = A . B^T of 4-bit operands (``fo_mx4_gemm``).

    A has M rows; B has N rows, or with ``row_ends`` (int32 [problems], on the
    device) ``problems * N``: problem p multiplies rows row_ends[p-1] ..
    row_ends[p] - 1 of A with its own N rows of B, stacked in order."""
    import torch
    if dtype not in _DTYPES:
        raise ValueError(f"dtype: {dtype!r}, expected one of {sorted(_DTYPES)}")
    device = _current(a_codes, "a_codes")
    if a_codes.dim() != 2 or b_codes.dim() != 2 or a_codes.shape[1] != b_codes.shape[1]:
        raise ValueError(f"codes: shapes {tuple(a_codes.shape)} and {tuple(b_codes.shape)} do not multiply")
    M, K = a_codes.shape[0], 2 * a_codes.shape[1]
    problems, ends = 1, 0
    if row_ends is not None:
        problems = row_ends.numel()
        if row_ends.dtype != torch.int32 or row_ends.dim() != 1 or problems < 1:
            raise ValueError("row_ends: expected int32 [problems]")
        ends = _tensor(row_ends, "row_ends", row_ends.shape, 4, device)
    if b_codes.shape[0] % problems:
        raise ValueError(f"b_codes: {b_codes.shape[0]} rows are not {problems} problems of equal size")
    N = b_codes.shape[0] // problems
    if out is None:
        out, = _new(stream, device, ((M, N), torch.bfloat16 if dtype == "bf16" else torch.float16))
    _check(_ops().fo_mx4_gemm(
        _tensor(a_codes, "a_codes", a_codes.shape, 1, device),
        _tensor(a_scales, "a_scales", mx4_shapes(M, K)[1], 1, device),
        _tensor(b_codes, "b_codes", b_codes.shape, 1, device),
        _tensor(b_scales, "b_scales", mx4_shapes(b_codes.shape[0], K)[1], 1, device),
        _tensor(out, "out", (M, N), 2, device), M, N, K, _DTYPES[dtype], problems, ends, _stream(stream)),
        "fo_mx4_gemm")
    return out
