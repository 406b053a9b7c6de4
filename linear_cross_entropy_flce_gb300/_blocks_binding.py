"""ctypes binding of include/flce_blocks.h: argument marshalling only.

Activations kept in 8 bits, alone and by the layer norm, and 4-bit floating point, made as the
operators' other calls are: the plain form through the extension _flce_ops, the general form here.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import Optional, Tuple

import torch

from ._ops_binding import (LayerNormResult, _c_int, _check, _declare, _device_of, _dtype_of, _f32, _fast,
                           _i32, _i64, _layer_norm_ws_bytes, _logits, _norm_params, _norm_rows, _output, _ptr,
                           _psize, _row_vector, _same_device, _size, _status, _stream, _vp, _workspace)

_packed_row_bytes = _declare("flce_packed_row_bytes", _c_int, _i64, ctypes.POINTER(_i64))
_pack = _declare("flce_pack_e4m3", _c_int, _vp, _i32, _i64, _i64, _i64, _vp, _vp)
_unpack = _declare("flce_unpack_e4m3", _c_int, _vp, _i64, _i64, _vp, _i32, _i64, _vp)
_layer_norm_packed = _declare("flce_layer_norm_packed", _c_int, _vp, _i32, _i64, _vp, _vp, _i32, _i64, _i64,
                              _f32, _vp, _i64, _vp, _vp, _vp, _vp)
_layer_norm_packed_backward = _declare(
    "flce_layer_norm_packed_backward", _c_int, _vp, _i32, _i64, _vp, _vp, _i32, _vp, _vp, _i64, _i64, _vp,
    _i64, _vp, _vp, _vp, _size, _vp)

_pi64 = ctypes.POINTER(_i64)
_fp4_sizes = _declare("flce_fp4_sizes", _c_int, _i64, _i64, _i32, _pi64, _psize)
_quantize_fp4 = _declare("flce_quantize_fp4", _c_int, _vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp)
_dequantize_fp4 = _declare("flce_dequantize_fp4", _c_int, _vp, _vp, _vp, _i64, _i64, _i32, _vp, _i32, _i64, _vp)
_linear_fp4 = _declare("flce_linear_fp4", _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp,
                       _i32, _i64, _i64, _vp, _vp)


@functools.lru_cache(maxsize=256)
def packed_row_bytes(D: int) -> int:
    """Bytes of the record of a row of D values."""
    size = _i64(0)
    _check(_packed_row_bytes(D, ctypes.byref(size)), "flce_packed_row_bytes")
    return int(size.value)


@dataclasses.dataclass
class PackedRows:
    """Values [*shape] in 8 bits: `data` holds a record per row (uint8 [rows, record bytes]): D
    E4M3 codes, padded to a multiple of 32, and a scale's exponent byte for each 32."""

    data: torch.Tensor
    shape: Tuple[int, ...]
    dtype: torch.dtype   # of what was packed

    @property
    def codes(self) -> torch.Tensor:
        """The E4M3 codes, uint8 [rows, D], a view."""
        return self.data[:, :self.shape[-1]]

    @property
    def scales(self) -> torch.Tensor:
        """e + 127 of each block's scale 2^e (255: the block is NaN), uint8 [rows, blocks], a view."""
        blocks = -(-self.shape[-1] // 32)
        return self.data[:, 32 * blocks:33 * blocks]


def _records(packed: PackedRows, dev) -> Tuple[int, int]:
    """(rows, D) of packed rows on dev."""
    D = packed.shape[-1]
    rows = 1
    for n in packed.shape[:-1]:
        rows *= n
    _same_device(packed.data, dev, "packed")
    if packed.data.dtype != torch.uint8 or tuple(packed.data.shape) != (rows, packed_row_bytes(D)) \
            or not packed.data.is_contiguous():
        raise ValueError("packed does not hold a record for each row")
    return rows, D


def _record_output(out, N, D, dev):
    if out is None:
        return torch.empty((N, packed_row_bytes(D)), dtype=torch.uint8, device=dev)
    _same_device(out, dev, "out")
    if out.dtype != torch.uint8 or tuple(out.shape) != (N, packed_row_bytes(D)) or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 tensor of a record for each row")
    return out


def pack_e4m3(x, *, out=None, stream=None) -> PackedRows:
    """x [..., D] (fp32 or bf16) in 8 bits, E4M3 with a power-of-two scale for each 32 values of
    a row, via flce_pack_e4m3. `out` may hold the records (uint8 [rows, packed_row_bytes(D)])."""
    if out is None and stream is None:
        data = _fast.pack_e4m3(x)
        if data is not None:
            return PackedRows(data, tuple(x.shape), x.dtype)
    dev = _device_of(x, "x")
    code = _dtype_of(x, "x")
    raw, ctx = _stream(stream, dev)
    with ctx:
        r, N, D, ld = _norm_rows(x, "x")
        data = _record_output(out, N, D, dev)
    _check(_pack(r.data_ptr(), code, ld, N, D, data.data_ptr(), raw), "flce_pack_e4m3")
    return PackedRows(data, tuple(x.shape), x.dtype)


def unpack_e4m3(packed: PackedRows, *, dtype: Optional[torch.dtype] = None, out=None, stream=None):
    """The values that packed rows stand for, as `dtype` (the packed tensor's own by default) or
    into `out`, via flce_unpack_e4m3."""
    if out is None and stream is None:
        r = _fast.unpack_e4m3(packed.data, packed.shape, packed.dtype if dtype is None else dtype)
        if r is not None:
            return r
    dev = _device_of(packed.data, "packed")
    N, D = _records(packed, dev)
    raw, ctx = _stream(stream, dev)
    if out is None:
        with ctx:
            out = torch.empty(packed.shape, dtype=packed.dtype if dtype is None else dtype, device=dev)
    else:
        _same_device(out, dev, "out")
        if tuple(out.shape) != tuple(packed.shape) or not out.is_contiguous() or dtype not in (None, out.dtype):
            raise ValueError("out must be a contiguous tensor of the packed shape and the dtype asked for")
    _check(_unpack(packed.data.data_ptr(), N, D, out.data_ptr(), _dtype_of(out, "the result"), D, raw),
           "flce_unpack_e4m3")
    return out


def layer_norm_packed(x, weight=None, bias=None, *, eps: float = 1e-5, out: Optional[dict] = None,
                      stream=None) -> Tuple[LayerNormResult, PackedRows]:
    """layer_norm of x, and x in 8 bits for layer_norm_packed_backward, via
    flce_layer_norm_packed. `out` may hold preallocated "y" (x's shape; it may be x), "mean",
    "rstd" ([N]) and "packed" (uint8 [N, packed_row_bytes(D)])."""
    if out is None and stream is None:
        r = _fast.layer_norm_packed(x, weight, bias, eps)
        if r is not None:
            return LayerNormResult(*r[:3]), PackedRows(r[3], tuple(x.shape), x.dtype)
    dev = _device_of(x, "x")
    code = _dtype_of(x, "x")
    raw, ctx = _stream(stream, dev)
    with ctx:
        r, N, D, ld = _norm_rows(x, "x")
        wcode = _norm_params(weight, bias, D, dev)
        y = _output(out, "y", x.shape, x.dtype, dev)
        mean = _output(out, "mean", (N,), torch.float32, dev)
        rstd = _output(out, "rstd", (N,), torch.float32, dev)
        data = _record_output(out.get("packed") if out else None, N, D, dev)
    _check(_layer_norm_packed(r.data_ptr(), code, ld, _ptr(weight), _ptr(bias), wcode, N, D, eps, y.data_ptr(), D,
                              mean.data_ptr(), rstd.data_ptr(), data.data_ptr(), raw), "flce_layer_norm_packed")
    return LayerNormResult(y, mean, rstd), PackedRows(data, tuple(x.shape), x.dtype)


def layer_norm_packed_backward(dy, packed: PackedRows, weight, result, *, need_dx: bool = True,
                               need_dweight: bool = True, need_dbias: bool = True, out: Optional[dict] = None,
                               workspace=None, stream=None):
    """(dx, dweight, dbias) of a layer_norm_packed call from its packed input, with h = (the
    packed value - mean) rstd, via flce_layer_norm_packed_backward; else as layer_norm_backward."""
    if out is None and workspace is None and stream is None and dy.dtype == packed.dtype:
        r = _fast.layer_norm_packed_backward(dy, packed.data, packed.shape, weight, result.mean, result.rstd,
                                             need_dx, need_dweight, need_dbias)
        if r is not None:
            return r
    dev = _device_of(dy, "dy")
    code = _dtype_of(dy, "dy")
    if dy.dtype != packed.dtype or tuple(dy.shape) != tuple(packed.shape):
        raise ValueError("dy must have the packed tensor's shape and dtype")
    N, D = _records(packed, dev)
    raw, ctx = _stream(stream, dev)
    with ctx:
        g, _, _, ldg = _norm_rows(dy, "dy")
        wcode = _norm_params(weight, None, D, dev)
        mean = _row_vector(result.mean, N, dev, "mean")
        rstd = _row_vector(result.rstd, N, dev, "rstd")
        wtype = weight.dtype if weight is not None else torch.float32
        dx = _output(out, "dx", dy.shape, dy.dtype, dev) if need_dx else None
        dw = _output(out, "dweight", (D,), wtype, dev) if need_dweight else None
        db = _output(out, "dbias", (D,), wtype, dev) if need_dbias else None
        ws = None
        if need_dweight or need_dbias:
            ws = _workspace(workspace, _layer_norm_ws_bytes(N, D), dev)
    _check(_layer_norm_packed_backward(
        g.data_ptr(), code, ldg, packed.data.data_ptr(), _ptr(weight), wcode, mean.data_ptr(), rstd.data_ptr(), N,
        D, _ptr(dx), D, _ptr(dw), _ptr(db), _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0, raw),
        "flce_layer_norm_packed_backward")
    return dx, dw, db


# ---- 4-bit floating point --------------------------------------------------------------------

FP4_FORMATS = {"mxfp4": 0, "nvfp4": 1}
_FP4_BLOCK = {"mxfp4": 32, "nvfp4": 16}


def _fp4_code(format: str) -> int:
    code = FP4_FORMATS.get(format)
    if code is None:
        raise ValueError(f"format must be one of {', '.join(FP4_FORMATS)}, not {format!r}")
    return code


@functools.lru_cache(maxsize=256)
def _fp4_bytes(N: int, D: int, code: int) -> Tuple[int, int]:
    row, scales = _i64(0), _size(0)
    _check(_fp4_sizes(N, D, code, ctypes.byref(row), ctypes.byref(scales)), "flce_fp4_sizes")
    return int(row.value), int(scales.value)


def _fp4_groups(D: int, format: str) -> int:
    """Groups of four neighbouring blocks of a row, padded to whole 256 values."""
    return -(-D // 256) * (64 // _FP4_BLOCK[format])


@dataclasses.dataclass
class Fp4Matrix:
    """Values [*shape] in 4-bit floating point, as the tensor cores read them: `codes` uint8 [rows,
    code bytes], two E2M1 codes to a byte; `scales` uint8, the blocks' scales in the tiled
    order of flce_blocks.h; `row_scales` fp32 [rows] (nvfp4) or None."""

    codes: torch.Tensor
    scales: torch.Tensor
    row_scales: Optional[torch.Tensor]
    shape: Tuple[int, ...]
    format: str

    def block_scales(self) -> torch.Tensor:
        """The blocks' scale bytes row by row, uint8 [rows, blocks], a copy."""
        N, D = self.codes.shape[0], self.shape[-1]
        blocks = -(-D // _FP4_BLOCK[self.format])
        tiles, groups = -(-N // 128), _fp4_groups(D, self.format)
        t = self.scales.view(tiles, groups, 32, 4, 4).permute(0, 3, 2, 1, 4)   # tile, r / 32, r % 32, group, block
        return t.reshape(tiles * 128, 4 * groups)[:N, :blocks].contiguous()

    @classmethod
    def from_rows(cls, codes, block_scales, row_scales=None, *, width: Optional[int] = None,
                  format: str = "nvfp4") -> "Fp4Matrix":
        """A matrix [N, width] of codes and scales that lie row by row, as checkpoints hold them:
        codes uint8 [N, ceil(width / 2)] (the first of two in the low bits), block_scales uint8
        or float8 [N, blocks] (nvfp4: not negative), and for nvfp4 row_scales, one value or [N] (1 if None)."""
        code = _fp4_code(format)
        if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_cuda:
            raise TypeError("codes must be a [N, bytes] uint8 CUDA tensor")
        N, D = codes.shape[0], 2 * codes.shape[1] if width is None else int(width)
        blocks = -(-D // _FP4_BLOCK[format])
        if codes.shape[1] != (D + 1) // 2 or tuple(block_scales.shape) != (N, blocks) \
                or block_scales.element_size() != 1:
            raise ValueError("codes and block_scales must hold ceil(width / 2) bytes and one byte per block of a row")
        row, _ = _fp4_bytes(N, D, code)
        wide = codes.new_zeros((N, row))
        wide[:, :codes.shape[1]] = codes
        if D % 2:
            wide[:, codes.shape[1] - 1] &= 15
        tiles, groups = -(-N // 128), _fp4_groups(D, format)
        full = codes.new_zeros((tiles * 128, 4 * groups))
        full[:N, :blocks] = block_scales.view(torch.uint8)
        scales = full.view(tiles, 4, 32, groups, 4).permute(0, 3, 2, 1, 4).reshape(-1)
        if format == "nvfp4":
            given = torch.as_tensor(1.0 if row_scales is None else row_scales, dtype=torch.float32, device=codes.device)
            if given.numel() != 1 and tuple(given.shape) != (N,):
                raise ValueError("row_scales must be one value or [N]")
            row_scales = given.reshape(-1).expand(N).clone(memory_format=torch.contiguous_format)
        elif row_scales is not None:
            raise ValueError("mxfp4 has no row scales")
        return cls(wide, scales, row_scales, (N, D), format)


def _fp4_matrix(m: Fp4Matrix, dev, name: str):
    """(rows, D, format code) of a matrix on dev."""
    D = m.shape[-1]
    rows = 1
    for n in m.shape[:-1]:
        rows *= n
    code = _fp4_code(m.format)
    row, size = _fp4_bytes(rows, D, code)
    for t, what, dtype, shape in ((m.codes, "codes", torch.uint8, (rows, row)), (m.scales, "scales", torch.uint8, (size,)),
                                  (m.row_scales, "row_scales", torch.float32, (rows,))):
        if what == "row_scales" and not code:
            continue
        _same_device(t, dev, f"{name}.{what}")
        if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name}.{what} must be a contiguous {dtype} tensor of shape {shape}")
    return rows, D, code


def quantize_fp4(x, *, format: str = "nvfp4", stream=None) -> Fp4Matrix:
    """x [..., D] (fp32 or bf16) in 4-bit floating point, "nvfp4" (blocks of 16 with E4M3 scales and
    a power of two for each row) or "mxfp4" (blocks of 32 with powers of two), via flce_quantize_fp4."""
    code = _fp4_code(format)
    if stream is None:
        r = _fast.quantize_fp4(x, code)
        if r is not None:
            return Fp4Matrix(*r, tuple(x.shape), format)
    dev = _device_of(x, "x")
    dtype = _dtype_of(x, "x")
    raw, ctx = _stream(stream, dev)
    with ctx:
        r, N, D, ld = _norm_rows(x, "x")
        row, size = _fp4_bytes(N, D, code)
        codes = torch.empty((N, row), dtype=torch.uint8, device=dev)
        scales = torch.empty(size, dtype=torch.uint8, device=dev)
        rows = torch.empty(N, dtype=torch.float32, device=dev) if code else None
    _check(_quantize_fp4(r.data_ptr(), dtype, ld, N, D, code, codes.data_ptr(), scales.data_ptr(), _ptr(rows), raw),
           "flce_quantize_fp4")
    return Fp4Matrix(codes, scales, rows, tuple(x.shape), format)


def dequantize_fp4(m: Fp4Matrix, *, dtype: torch.dtype = torch.float32, out=None, stream=None):
    """The values of a 4-bit matrix, as `dtype` (fp32 or bf16) or into `out`, via
    flce_dequantize_fp4."""
    if out is None and stream is None:
        r = _fast.dequantize_fp4(m.codes, m.scales, m.row_scales, m.shape, _fp4_code(m.format), dtype)
        if r is not None:
            return r
    dev = _device_of(m.codes, "codes")
    N, D, code = _fp4_matrix(m, dev, "the matrix")
    raw, ctx = _stream(stream, dev)
    if out is None:
        with ctx:
            out = torch.empty(m.shape, dtype=dtype, device=dev)
    else:
        _same_device(out, dev, "out")
        if tuple(out.shape) != tuple(m.shape) or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor of the matrix's shape")
    _check(_dequantize_fp4(m.codes.data_ptr(), m.scales.data_ptr(), _ptr(m.row_scales), N, D, code, out.data_ptr(),
                           _dtype_of(out, "the result"), D, raw), "flce_dequantize_fp4")
    return out


def linear_fp4(h: Fp4Matrix, w: Fp4Matrix, *, dtype: torch.dtype = torch.bfloat16, out=None, status=None,
               timeout_ns: int = 0, stream=None):
    """[*h.shape[:-1], V] of two 4-bit matrices h [..., D] and w [V, D] of one format: h w^T, accumulated
    in fp32 on the block-scaled tensor cores and rounded once to `dtype` (fp32 or bf16), via
    flce_linear_fp4. `out` may be preallocated, its rows any distance apart. No gradient."""
    if out is None and status is None and not timeout_ns and stream is None and h.format == w.format:
        r = _fast.linear_fp4(h.codes, h.scales, h.row_scales, h.shape, w.codes, w.scales, w.row_scales, w.shape,
                             _fp4_code(h.format), dtype)
        if r is not None:
            return r
    dev = _device_of(h.codes, "h")
    N, D, code = _fp4_matrix(h, dev, "h")
    V, Dw, wcode = _fp4_matrix(w, dev, "w")
    if code != wcode:
        raise ValueError("h and w must have one format")
    if D != Dw or len(w.shape) != 2:
        raise ValueError("h must be [..., D] and w [V, D]")
    raw, ctx = _stream(stream, dev)
    shape = (*h.shape[:-1], V)
    if out is None:
        with ctx:
            out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _same_device(out, dev, "out")
        if tuple(out.shape) != shape or out.dim() != 2 and not out.is_contiguous():
            raise ValueError(f"out must be of shape {shape}, and contiguous if not a matrix")
    flat = out if out.dim() == 2 else out.view(-1, V)
    _, _, ldy = _logits(flat, "out")
    _check(_linear_fp4(h.codes.data_ptr(), h.scales.data_ptr(), _ptr(h.row_scales), w.codes.data_ptr(),
                       w.scales.data_ptr(), _ptr(w.row_scales), N, D, V, code, out.data_ptr(),
                       _dtype_of(out, "the result"), ldy, int(timeout_ns), _status(status, dev), raw),
           "flce_linear_fp4")
    return out
