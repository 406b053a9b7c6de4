"""ctypes binding of include/flce_embed.h: argument marshalling only.

Embedding lookup and the gradient of its table, made as the operators' other calls are: the
plain form through the extension _flce_ops, the general form here.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._binding import ignore_id
from ._ops_binding import (_c_int, _check, _declare, _device_of, _dtype_of, _f32, _fast, _i32, _i64,
                           _logits, _norm_rows, _ptr, _psize, _same_device, _size, _status, _stream,
                           _vp, _workspace)

_embedding = _declare("flce_embedding", _c_int, _vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _i32,
                      _vp, _i32, _i64, _vp, _vp)
_embedding_ws = _declare("flce_embedding_backward_workspace_size", _c_int, _i64, _i64, _i64, _psize)
_embedding_backward = _declare(
    "flce_embedding_backward", _c_int, _vp, _i32, _i64, _vp, _i64, _i64, _i64, _f32, _i32, _vp, _i32,
    _i64, _i32, _vp, _size, _vp)


def _ids(tokens, dev):
    """int32 tokens of any shape, dense in their order."""
    _same_device(tokens, dev, "tokens")
    if tokens.dtype != torch.int32:
        raise TypeError("tokens must be int32")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return tokens


def embedding(weight, tokens, *, scale: float = 1.0, ignore_index: int = -100,
              dtype: Optional[torch.dtype] = None, out=None, status=None, stream=None):
    """scale * weight[tokens], [*tokens.shape, D], via flce_embedding: weight [V, D] (fp32 or
    bf16, any row stride), tokens int32 of any shape. Rows of ignore_index are 0. The result
    has `dtype` (the weight's by default), or goes to `out`. `status`, an int32 tensor the
    caller zeroed, receives device errors (a token out of range, whose row is NaN)."""
    if out is None and status is None and stream is None:
        r = _fast.embedding(weight, tokens, scale, ignore_index, dtype)
        if r is not None:
            return r
    dev = _device_of(weight, "weight")
    wcode = _dtype_of(weight, "weight")
    V, D, ldw = _logits(weight, "weight")
    ids = _ids(tokens, dev)
    raw, ctx = _stream(stream, dev)
    if out is None:
        with ctx:
            out = torch.empty((*ids.shape, D), dtype=weight.dtype if dtype is None else dtype, device=dev)
    else:
        _same_device(out, dev, "out")
        if tuple(out.shape) != (*ids.shape, D) or not out.is_contiguous() or dtype not in (None, out.dtype):
            raise ValueError("out must be a contiguous [*tokens.shape, D] tensor of the dtype asked for")
    code = _dtype_of(out, "the result")
    _check(_embedding(weight.data_ptr(), wcode, ldw, ids.data_ptr(), ids.numel(), V, D, float(scale),
                      ignore_id(ignore_index), out.data_ptr(), code, D, _status(status, dev), raw), "flce_embedding")
    return out


@functools.lru_cache(maxsize=256)
def _embedding_ws_bytes(N, V, D) -> int:
    size = _size(0)
    _check(_embedding_ws(N, V, D, ctypes.byref(size)), "flce_embedding_backward_workspace_size")
    return int(size.value)


def embedding_backward_workspace_size(N: int, V: int, D: int) -> int:
    """Workspace bytes of embedding_backward for N tokens and a [V, D] table."""
    return _embedding_ws_bytes(N, V, D)


def embedding_backward(dy, tokens, rows: int, *, scale: float = 1.0, ignore_index: int = -100,
                       dtype: Optional[torch.dtype] = None, out=None, accumulate: bool = False,
                       workspace=None, stream=None):
    """Gradient [rows, D] of the table of an embedding call, from dy [*tokens.shape, D] (fp32
    or bf16), via flce_embedding_backward: every row is written (zeros for ids without
    tokens), as `dtype` (dy's by default) or into `out`. With `accumulate` it is added to
    `out` instead, where only rows of tokens are touched."""
    if out is None and not accumulate and workspace is None and stream is None:
        r = _fast.embedding_backward(dy, tokens, rows, scale, ignore_index, dtype)
        if r is not None:
            return r
    dev = _device_of(dy, "dy")
    code = _dtype_of(dy, "dy")
    ids = _ids(tokens, dev)
    if dy.shape[:-1] != ids.shape:
        raise ValueError("dy must be [*tokens.shape, D]")
    if accumulate and out is None:
        raise ValueError("accumulate needs the table to add to, out")
    raw, ctx = _stream(stream, dev)
    with ctx:
        g, N, D, ldg = _norm_rows(dy, "dy")
        if out is None:
            out = torch.empty((rows, D), dtype=dy.dtype if dtype is None else dtype, device=dev)
        else:
            _same_device(out, dev, "out")
            if tuple(out.shape) != (rows, D) or dtype not in (None, out.dtype):
                raise ValueError("out must be a [rows, D] tensor of the dtype asked for")
        wcode = _dtype_of(out, "the gradient")
        _, _, ldw = _logits(out, "out")
        ws = _workspace(workspace, _embedding_ws_bytes(N, rows, D), dev)
    _check(_embedding_backward(g.data_ptr(), code, ldg, _ptr(ids), N, rows, D, float(scale),
                               ignore_id(ignore_index), out.data_ptr(), wcode, ldw, int(accumulate),
                               ws.data_ptr(), ws.numel() * ws.element_size(), raw),
           "flce_embedding_backward")
    return out
