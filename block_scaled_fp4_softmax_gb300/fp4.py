"""Thin ctypes binding over the C ABI in include/fp4.h.

The dense part of a decoder layer in block-scaled FP4: quantisation, products of
two FP4 matrices, SwiGLU and the norms around a residual sum.  As in :mod:`.moe`,
each function carries the C entry point's name, checks types and devices, allocates
what the caller does not pass, and hands device pointers plus the current CUDA
stream to the library.  The operands' device has to be the current one.

Rows are 2-D tensors whose columns are contiguous; they may be strided views
(``include/fp4.h`` states the alignment).
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from . import moe as _moe
from .moe import DEV_TIMEOUT, MoeError, _check  # noqa: F401

NVFP4 = _moe.FMT_NVFP4
MXFP4 = _moe.FMT_MXFP4

EXPORTS = (
    "fp4_scale_bytes",
    "fp4_tile_scales",
    "fp4_quantize",
    "fp4_dequantize",
    "fp4_swiglu",
    "fp4_block_norm",
    "fp4_linear",
    "fp4_linear_rows_workspace",
    "fp4_linear_rows",
)

_BLOCK = {NVFP4: 16, MXFP4: 32}
_bf16, _f16, _f32, _u8, _i32 = torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int32
_TYPES = {_bf16: 0, _f16: 1, _f32: 2}
_SHORT = {_bf16: 0, _f16: 1}


class _MatrixStruct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("format", ctypes.c_int32)]


_vp, _i, _ll, _d, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_double, ctypes.c_size_t

# matrices go by their address, a plain number
_SIGS = {
    "fp4_scale_bytes": (_sz, [_i, _i, _i]),
    "fp4_tile_scales": (_i, [_vp, _i, _i, _i, _vp, _vp]),
    "fp4_quantize": (_i, [_vp, _ll, _i, _vp, _vp]),
    "fp4_dequantize": (_i, [_vp, _vp, _ll, _i, _vp]),
    "fp4_swiglu": (_i, [_vp, _ll, _vp, _ll, _i, _i, _i, _vp, _ll, _i, _vp, _vp]),
    "fp4_block_norm": (_i, [_vp, _ll, _i, _vp, _ll, _i, _vp, _vp, _ll, _i, _d, _vp, _d, _i, _i, _vp, _ll, _vp, _ll, _i,
                            _vp, _vp]),
    "fp4_linear": (_i, [_vp, _vp, _vp, _vp, _ll, _i, _vp, _vp]),
    "fp4_linear_rows_workspace": (_sz, [_vp, _i]),
    "fp4_linear_rows": (_i, [_vp, _ll, _i, _i, _vp, _vp, _vp, _ll, _i, _vp, _sz, _vp, _vp]),
}

_LIB = None


def load():
    """The library of :func:`.moe.load` with this module's signatures set."""
    global _LIB
    if _LIB is None:
        lib = _moe.load()
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


# ---------------------------------------------------------------------------
# Checks.  They run on every call of a decode step, so each is a handful of
# attribute reads; the words for a refusal are only put together when there is one.
# ---------------------------------------------------------------------------

_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice
_HERE = contextlib.nullcontext()
_empty = torch.empty


def _wrong_device(index):
    raise MoeError(f"the operands are on cuda:{index}, cuda:{_current()} is current")


def _index(t, name):
    """CUDA device of an operand, which has to be the current one: a launch goes there.
    Any other is refused before anything else is done."""
    try:
        index = t.get_device()
    except AttributeError:
        index = -1
    if index < 0:
        raise MoeError(f"{name} must be a CUDA tensor")
    if _current() != index:
        _wrong_device(index)
    return index


def _of(m, name):
    """Device of a matrix, which has to be the current one."""
    if m.__class__ is not Fp4Matrix:
        raise MoeError(f"{name} must be an FP4 matrix (fp4_matrix, fp4_empty), got {type(m).__name__}")
    if _current() != m.index:
        _wrong_device(m.index)
    return m.index


def _on(stream, index):
    """Handle of the stream to launch on."""
    if stream is None:
        return _raw_stream(index)
    if stream.device_index != index:
        raise MoeError(f"the operands are on cuda:{index}, the stream on cuda:{stream.device_index}")
    return stream.cuda_stream


def _elsewhere(stream):
    """Context for allocating on the stream the call runs on, so that the
    allocator never hands the memory to another stream while the call uses it."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _rows(t, name, index, shape=None, types=_TYPES):
    """Address, stride and type of a [rows, cols] tensor with contiguous columns."""
    try:
        rows, one = t.stride()
        if t.get_device() == index and (one == 1 or t.shape[1] == 1) and (shape is None or t.shape == shape):
            return t.data_ptr(), rows, types[t.dtype]
    except (AttributeError, TypeError, ValueError, KeyError):
        pass
    raise MoeError(f"{name} must be a {list(shape) if shape else '[rows, cols]'} tensor of "
                   f"{', '.join(map(str, types))} on cuda:{index}, columns contiguous")


def _array(t, name, shape, dtype, index):
    """Address of a contiguous tensor of just this shape and type."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
            return t.data_ptr()
    except (AttributeError, TypeError):
        pass
    raise MoeError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")


def _matrix(m, name, index, shape, format=None):
    """Address of a matrix's C description."""
    if (m.__class__ is Fp4Matrix and m.shape == shape and m.index == index
            and (format is None or m.format == format)):
        return m.at
    raise MoeError(f"{name} must be a {list(shape)} FP4 matrix{'' if format is None else f' of format {format}'} "
                   f"on cuda:{index}, got {m!r}")


# ---------------------------------------------------------------------------
# Matrices
# ---------------------------------------------------------------------------

class Fp4Matrix:
    """A matrix in FP4: the C description plus the tensors it points into, which
    it keeps alive.  ``codes`` [rows, cols / 2] uint8, ``scales`` uint8 in the
    layout that products read, ``row_scale`` [rows] float32 or None: the description
    holds their addresses, so they are written into, never replaced."""

    def __init__(self, codes, scales, row_scale, rows, cols, format):
        _check_shape(rows, cols, format)
        index = codes.get_device()
        at = (_array(codes, "codes", (rows, cols // 2), _u8, index),
              _array(scales, "scales", (_scale_bytes(rows, cols, format),), _u8, index),
              None if row_scale is None else _array(row_scale, "row_scale", (rows,), _f32, index))
        self._parts = codes, scales, row_scale
        self.rows, self.cols, self.format, self.shape = rows, cols, format, (rows, cols)
        self.device, self.index = codes.device, index
        self.struct = _MatrixStruct(*at, rows, cols, format)
        self.at = ctypes.addressof(self.struct)

    codes = property(lambda self: self._parts[0])
    scales = property(lambda self: self._parts[1])
    row_scale = property(lambda self: self._parts[2])

    def __reduce__(self):  # a copy, or a saved one, has a description of its own tensors
        return Fp4Matrix, (*self._parts, self.rows, self.cols, self.format)

    def __repr__(self):
        return f"Fp4Matrix({self.rows} x {self.cols}, {'NVFP4' if self.format == NVFP4 else 'MXFP4'}, {self.device})"


def fp4_scale_bytes(rows: int, cols: int, format: int) -> int:
    """Bytes of the laid-out scales of a matrix."""
    if not (0 <= rows < 1 << 31 and 0 <= cols < 1 << 31):
        return 0
    return int(load().fp4_scale_bytes(rows, cols, format))


def _scale_bytes(rows, cols, format):
    """fp4_scale_bytes of a shape that has been checked, without a call."""
    span = 4 * _BLOCK[format]
    return (rows + 127) // 128 * ((cols + span - 1) // span) * 512


def _check_shape(rows, cols, format):
    if format not in _BLOCK or not 0 <= rows <= 1 << 24 or not 32 <= cols <= 32768 or cols % 32:
        raise MoeError(f"no FP4 matrix has the shape {rows} x {cols} in format {format}: cols is a multiple of 32 "
                       f"from 32 to 32768, rows at most 2^24")


def fp4_empty(rows: int, cols: int, format: int = NVFP4, device=None, stream=None) -> Fp4Matrix:
    """A matrix whose elements are still to be written."""
    _check_shape(rows, cols, format)
    device = torch.device("cuda", _current()) if device is None else torch.device(device)
    with _elsewhere(stream):
        codes = _empty((rows, cols // 2), dtype=_u8, device=device)
        scales = _empty(_scale_bytes(rows, cols, format), dtype=_u8, device=device)
        row_scale = _empty(rows, dtype=_f32, device=device) if format == NVFP4 else None
    return Fp4Matrix(codes, scales, row_scale, rows, cols, format)


def fp4_tile_scales(scales, cols: int, format: int, tiled=None, stream=None):
    """Row-major block scales [rows, cols / 16 (MXFP4: 32)] uint8, as checkpoints
    and expert records hold them, in the layout that products read."""
    index = _index(scales, "scales")
    on = _on(stream, index)
    rows = scales.shape[0] if scales.dim() == 2 else -1
    _check_shape(rows, cols, format)
    at = _array(scales, "scales", (rows, cols // _BLOCK[format]), _u8, index)
    size = _scale_bytes(rows, cols, format)
    if tiled is None:
        with _elsewhere(stream):
            tiled = _empty(size, dtype=_u8, device=scales.device)
    _check(load().fp4_tile_scales(at, rows, cols, format, _array(tiled, "tiled", (size,), _u8, index), on),
           "fp4_tile_scales")
    return tiled


def fp4_matrix(codes, scales, row_scale=None, format: int = NVFP4, stream=None) -> Fp4Matrix:
    """A matrix of a checkpoint's or record's parts: codes [rows, cols / 2] uint8
    (kept, not copied), scales [rows, cols / 16 (MXFP4: 32)] uint8 row-major (laid
    out anew), row_scale [rows] float32 or None."""
    index = _index(codes, "codes")
    if codes.dim() != 2:
        raise MoeError("codes must be [rows, cols / 2]")
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    _check_shape(rows, cols, format)
    _array(codes, "codes", (rows, cols // 2), _u8, index)
    if row_scale is not None:
        _array(row_scale, "row_scale", (rows,), _f32, index)
    return Fp4Matrix(codes, fp4_tile_scales(scales, cols, format, stream=stream), row_scale, rows, cols, format)


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def fp4_quantize(x, format: int = NVFP4, out: Fp4Matrix | None = None, stream=None) -> Fp4Matrix:
    """x [rows, cols] of bfloat16, float16 or float32 as an FP4 matrix."""
    index = _index(x, "x")
    on = _on(stream, index)
    at, stride, kind = _rows(x, "x", index)
    if out is None:
        out = fp4_empty(*x.shape, format, x.device, stream)
    rc = (_LIB or load()).fp4_quantize(at, stride, kind, _matrix(out, "out", index, x.shape, format), on)
    if rc:
        _check(rc, "fp4_quantize")
    return out


def fp4_dequantize(m: Fp4Matrix, dtype=torch.bfloat16, out=None, stream=None):
    """The values of m's elements, [rows, cols] of dtype (or out's type)."""
    index = _of(m, "m")
    on = _on(stream, index)
    out, to = _result(m.shape, dtype, m.device, stream) if out is None else (out, _rows(out, "out", index, m.shape))
    rc = (_LIB or load()).fp4_dequantize(m.at, *to, on)
    if rc:
        _check(rc, "fp4_dequantize")
    return out


_NOTHING = (None, 0, 0)


def _targets(shape, t, dtype, format, out, matrix, index, stream, names):
    """What a call writes, made where it is wanted and not given: the 16-bit output, its
    description, the FP4 output and its address."""
    to, at = _NOTHING, None
    if out is None:
        if dtype is not None:
            if dtype not in _SHORT:
                raise MoeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
            out, to = _result(shape, dtype, t.device, stream)
    else:
        to = _rows(out, names[0], index, shape, _SHORT)
    if matrix is None and format is not None:
        matrix = fp4_empty(*shape, format, t.device, stream)
    if matrix is not None:
        at = _matrix(matrix, names[1], index, shape, format)
    elif out is None:
        raise MoeError(f"neither {names[0]} nor {names[1]} is wanted")
    return out, to, matrix, at


def fp4_swiglu(gate, up, dtype=torch.bfloat16, format: int | None = None, out=None, matrix: Fp4Matrix | None = None,
               stream=None):
    """SiLU(gate) * up, [rows, cols] each.  Returns (out of dtype or None, FP4
    matrix of format or None): dtype = None and format = None leave theirs away.
    out may be gate or up, where its elements are as wide."""
    index = _index(gate, "gate")
    on = _on(stream, index)
    g, g_stride, kind = _rows(gate, "gate", index)
    shape = gate.shape
    u, u_stride, other = _rows(up, "up", index, shape)
    if other != kind:
        raise MoeError(f"gate and up must be of one type, got {gate.dtype} and {up.dtype}")
    out, to, matrix, at = _targets(shape, gate, dtype, format, out, matrix, index, stream, ("out", "matrix"))
    rows, cols = shape
    rc = (_LIB or load()).fp4_swiglu(g, g_stride, u, u_stride, kind, rows, cols, *to, at, on)
    if rc:
        _check(rc, "fp4_swiglu")
    return out, matrix


def fp4_block_norm(r, y=None, post_weight=None, gate=None, scale: float = 1.0, weight=None, eps: float = 1e-6,
                   dtype=torch.bfloat16, format: int | None = None, r_out=None, out=None,
                   matrix: Fp4Matrix | None = None, stream=None):
    """r_out = r + scale * gate * norm(y; post_weight) and its norm(r_out; weight).

    r, y [rows, cols]; weights [cols] float32; gate [cols], [rows, cols] or [rows,
    1] of y's type.  r_out and out may be r, y or a [rows, cols] gate, where their
    elements are as wide.  Returns (r_out, norm of dtype or None, norm
    as an FP4 matrix of format or None); without y, r itself is r_out."""
    index = _index(r, "r")
    on = _on(stream, index)
    a = _rows(r, "r", index)
    shape = r.shape
    rows, cols = shape
    b, g, gate_stride, gate_cols, to, to_stride = _NOTHING, None, 0, 0, None, 0
    if y is None:
        if post_weight is not None or gate is not None or r_out is not None:
            raise MoeError("post_weight, gate and r_out go with y")
        r_out = r
    else:
        b = _rows(y, "y", index, shape)
        if gate is not None:
            g, gate_stride, gate_cols = _gate(gate, y, index, shape)
        if r_out is r:
            to, to_stride = a[:2]
        elif r_out is None:
            r_out, (to, to_stride, _) = _result(shape, r.dtype, r.device, stream)
        else:
            to, to_stride, kind = _rows(r_out, "r_out", index, shape)
            if kind != a[2]:
                raise MoeError(f"r_out must be of r's type, got {r_out.dtype} and {r.dtype}")
    post = None if post_weight is None else _array(post_weight, "post_weight", (cols,), _f32, index)
    w = None if weight is None else _array(weight, "weight", (cols,), _f32, index)
    out, h, matrix, at = _targets(shape, r, dtype, format, out, matrix, index, stream, ("out", "matrix"))
    rc = (_LIB or load()).fp4_block_norm(*a, *b, post, g, gate_stride, gate_cols, scale, w, eps, rows, cols, to,
                                         to_stride, *h, at, on)
    if rc:
        _check(rc, "fp4_block_norm")
    return r_out, out, matrix


def _gate(gate, y, index, shape):
    """Address, row stride and columns of a gate."""
    try:
        form = gate.shape
        if gate.dtype is y.dtype and gate.get_device() == index:
            if form == shape[1:] and gate.is_contiguous():
                return gate.data_ptr(), 0, shape[1]
            if form == shape and gate.stride(1) == 1:
                return gate.data_ptr(), gate.stride(0), shape[1]
            if form == (shape[0], 1):
                return gate.data_ptr(), gate.stride(0), 1
    except (AttributeError, TypeError):
        pass
    raise MoeError(f"gate must be a {list(shape[1:])}, {list(shape)} or {[shape[0], 1]} tensor of {y.dtype} on "
                   f"cuda:{index}, columns contiguous")


def _result(shape, dtype, device, stream):
    """A new output with its address, stride and type."""
    kind = _TYPES.get(dtype)
    if kind is None:
        raise MoeError(f"dtype must be one of {', '.join(map(str, _TYPES))}, got {dtype}")
    if stream is None:
        out = _empty(shape, dtype=dtype, device=device)
    else:
        with torch.cuda.stream(stream):
            out = _empty(shape, dtype=dtype, device=device)
    return out, (out.data_ptr(), shape[1], kind)


def fp4_linear(x: Fp4Matrix, w: Fp4Matrix, bias=None, dtype=torch.bfloat16, out=None, dev_status=None, stream=None):
    """x [tokens, cols] times w [features, cols], both in FP4 of one format, plus
    bias [features] float32: [tokens, features] of dtype (or out's type)."""
    index = _of(w, "w")
    on = _on(stream, index)
    _of(x, "x")
    if x.cols != w.cols or x.format != w.format:
        raise MoeError(f"x and w must have the same columns and format, got {x!r} and {w!r}")
    shape = (x.rows, w.rows)
    out, to = _result(shape, dtype, w.device, stream) if out is None else (out, _rows(out, "out", index, shape))
    rc = (_LIB or load()).fp4_linear(
        x.at, w.at, None if bias is None else _array(bias, "bias", (w.rows,), _f32, index), *to,
        None if dev_status is None else _array(dev_status, "dev_status", (1,), _i32, index), on)
    if rc:
        _check(rc, "fp4_linear")
    return out


def fp4_linear_rows_workspace(w: Fp4Matrix, rows: int):
    """A workspace for :func:`fp4_linear_rows` with up to `rows` rows."""
    _of(w, "w")
    if not 0 <= rows <= 1 << 24:
        raise MoeError(f"rows must be 0 to 2^24, got {rows}")
    n = int(load().fp4_linear_rows_workspace(w.at, rows))
    if n == 0:
        raise MoeError("fp4_linear_rows does not support this matrix")
    return torch.empty(n, dtype=_u8, device=w.device)


def fp4_linear_rows(x, w: Fp4Matrix, bias=None, dtype=torch.bfloat16, out=None, workspace=None, dev_status=None,
                    stream=None):
    """:func:`fp4_linear` of x [tokens, cols] of bfloat16, float16 or float32,
    quantised in w's format."""
    index = _of(w, "w")
    on = _on(stream, index)
    at, stride, kind = _rows(x, "x", index)
    T, cols = x.shape
    if cols != w.cols:
        raise MoeError(f"x must be [tokens, {w.cols}], got {list(x.shape)}")
    shape = (T, w.rows)
    out, to = _result(shape, dtype, w.device, stream) if out is None else (out, _rows(out, "out", index, shape))
    if workspace is None:
        with _elsewhere(stream):
            workspace = fp4_linear_rows_workspace(w, T)
    try:
        size = workspace.shape[-1]
    except (AttributeError, IndexError):
        raise MoeError("workspace must be a tensor with a shape") from None
    rc = (_LIB or load()).fp4_linear_rows(
        at, stride, kind, T, w.at, None if bias is None else _array(bias, "bias", (w.rows,), _f32, index),
        *to, _array(workspace, "workspace", (size,), _u8, index), size,
        None if dev_status is None else _array(dev_status, "dev_status", (1,), _i32, index), on)
    if rc:
        _check(rc, "fp4_linear_rows")
    return out
