"""ctypes binding of include/flce_blocks.h: argument marshalling only.

Activations kept in 8 bits, alone and by the layer norm, made as the operators' other calls are:
the plain form through the extension _flce_ops, the general form here.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import Optional, Tuple

import torch

from ._ops_binding import (LayerNormResult, _c_int, _check, _declare, _device_of, _dtype_of, _f32, _fast,
                           _i32, _i64, _layer_norm_ws_bytes, _norm_params, _norm_rows, _output, _ptr,
                           _row_vector, _same_device, _size, _stream, _vp, _workspace)

_packed_row_bytes = _declare("flce_packed_row_bytes", _c_int, _i64, ctypes.POINTER(_i64))
_pack = _declare("flce_pack_e4m3", _c_int, _vp, _i32, _i64, _i64, _i64, _vp, _vp)
_unpack = _declare("flce_unpack_e4m3", _c_int, _vp, _i64, _i64, _vp, _i32, _i64, _vp)
_layer_norm_packed = _declare("flce_layer_norm_packed", _c_int, _vp, _i32, _i64, _vp, _vp, _i32, _i64, _i64,
                              _f32, _vp, _i64, _vp, _vp, _vp, _vp)
_layer_norm_packed_backward = _declare(
    "flce_layer_norm_packed_backward", _c_int, _vp, _i32, _i64, _vp, _vp, _i32, _vp, _vp, _i64, _i64, _vp,
    _i64, _vp, _vp, _vp, _size, _vp)


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
