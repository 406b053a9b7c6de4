"""ctypes binding of include/flce_ops.h: argument marshalling only.

Log probabilities of given tokens (over logits, or straight from hidden states), layer
norm, and the global gradient norm with clipping. Every computation happens in the
library's CUDA kernels; PyTorch provides device memory and streams.

The plain form of a call (nothing preallocated, the current stream) is made by the
extension _flce_ops, which takes a third of the time on the host; it returns None, with
nothing enqueued, for what it does not take, and the general form below then serves the
call or says what is wrong with it. A CUDA error, which may come after a launch, is raised.
Without the extension (it is built for one PyTorch) the general form serves every call.

Each call takes an optional `stream` (a torch.cuda.Stream or a raw cudaStream_t; the
current stream by default). What a call allocates for itself belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools
import re
import warnings
from typing import Optional, Sequence

import torch

from ._binding import FLCE_OK, FLCEError, ignore_id, lib


class _NoExtension:
    """Takes no call: all of them go through the general form."""

    def __getattr__(self, name):
        return lambda *args: None


def _load_extension():
    """_flce_ops, if there is one for this PyTorch."""
    try:
        from . import _flce_ops as fast
        have = re.match(r"[\d.]*\d", torch.__version__).group()
        if fast.torch_version != have:
            raise ImportError(f"built for PyTorch {fast.torch_version}, not {have}")
    except ImportError as e:
        warnings.warn(f"without _flce_ops, calls take longer on the host: {e}", RuntimeWarning)
        return _NoExtension()
    fast.set_error_type(FLCEError)
    return fast


_fast = _load_extension()

MAX_TOP_K = 32

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f32 = ctypes.c_float
_size = ctypes.c_size_t


class LogprobOptions(ctypes.Structure):
    _fields_ = [
        ("ignore_index", _i32),
        ("top_k", _i32),
        ("temperature", _f32),
        ("dw_dtype", _i32),
        ("timeout_ns", _i64),
    ]


_opt = ctypes.POINTER(LogprobOptions)
_psize = ctypes.POINTER(_size)


def _declare(name, restype, *argtypes):
    f = getattr(lib, name)
    f.argtypes = list(argtypes)
    f.restype = restype
    return f


_c_int = ctypes.c_int
_declare("flce_default_logprob_options", None, _opt)
_token_logprobs = _declare("flce_token_logprobs", _c_int, _vp, _i32, _i64, _vp, _i64, _i64, _opt,
                           _vp, _vp, _vp, _vp, _vp, _vp, _vp)
_token_logprobs_backward = _declare(
    "flce_token_logprobs_backward", _c_int, _vp, _i32, _i64, _vp, _i64, _i64, _opt, _vp, _vp, _vp,
    _vp, _vp, _vp, _vp, _i64, _vp)
_linear_ws = _declare("flce_linear_logprobs_workspace_size", _c_int, _i64, _i64, _i64, _opt, _i32,
                      _psize)
_linear_token_logprobs = _declare("flce_linear_token_logprobs", _c_int, _vp, _vp, _vp, _i64, _i64,
                                  _i64, _opt, _vp, _vp, _vp, _vp, _vp, _vp, _size, _vp, _vp)
_linear_token_logprobs_backward = _declare(
    "flce_linear_token_logprobs_backward", _c_int, _vp, _vp, _vp, _i64, _i64, _i64, _opt, _vp, _vp,
    _vp, _vp, _vp, _vp, _vp, _vp, _vp, _size, _vp, _vp)
_layer_norm = _declare("flce_layer_norm", _c_int, _vp, _i32, _i64, _vp, _vp, _i32, _i64, _i64,
                       _f32, _vp, _i64, _vp, _vp, _vp)
_layer_norm_ws = _declare("flce_layer_norm_workspace_size", _c_int, _i64, _i64, _psize)
_layer_norm_backward = _declare(
    "flce_layer_norm_backward", _c_int, _vp, _i64, _vp, _i32, _i64, _vp, _i32, _vp, _vp, _i64,
    _i64, _vp, _i64, _vp, _vp, _vp, _size, _vp)
_clip_ws = _declare("flce_clip_grads_workspace_size", _c_int, _i64, _psize)
_clip_grads = _declare("flce_clip_grads", _c_int, _vp, _vp, _vp, _vp, _i64, _f32, _vp, _vp, _size,
                       _vp)

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(rc: int, where: str) -> None:
    if rc != FLCE_OK:
        raise FLCEError(rc, where)


def _device_of(t, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is not on the current CUDA device")
    return t.device


def _dtype_of(t, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, not {t.dtype}")
    return code


_NO_CONTEXT = contextlib.nullcontext()


def _stream(stream, dev):
    """(raw handle, context in which the call's own memory is allocated)."""
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream, _NO_CONTEXT
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _same_device(t, dev, name: str) -> None:
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")


def _tokens(tokens, N: int, dev) -> Optional[int]:
    if tokens is None:
        return None
    _same_device(tokens, dev, "tokens")
    if tokens.dtype != torch.int32:
        raise TypeError("tokens must be int32")
    if tokens.dim() != 1 or tokens.shape[0] != N or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous [N] tensor")
    return tokens.data_ptr()


def _row_vector(t, N: int, dev, name: str):
    """A per-row fp32 vector as a contiguous tensor (gradients may come expanded)."""
    if t is None:
        return None
    _same_device(t, dev, name)
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.dim() != 1 or t.shape[0] != N:
        raise ValueError(f"{name} must have one value for each row")
    return t if t.is_contiguous() else t.contiguous()


def _output(out, key, shape, dtype, dev):
    """out[key] if the caller gave it (checked), else a new tensor."""
    t = out.get(key) if out else None
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if t.device != dev or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"out[{key!r}] must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}")
    return t


def _workspace(workspace, need: int, dev):
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _same_device(workspace, dev, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _status(status, dev) -> Optional[int]:
    if status is None:
        return None
    if status.device != dev or status.dtype != torch.int32 or status.numel() != 1:
        raise ValueError("status must be an int32 CUDA tensor of one element")
    return status.data_ptr()


def _options(ignore_index, top_k, temperature, dw_dtype=0, timeout_ns=0) -> LogprobOptions:
    return LogprobOptions(ignore_id(ignore_index), int(top_k), float(temperature), dw_dtype,
                          int(timeout_ns))


# ---- log probabilities -----------------------------------------------------------------------


@dataclasses.dataclass
class TokenLogprobs:
    """Per row: the token's log probability (0 without a token), the entropy, the
    log-sum-exp (all of the logits divided by the temperature), and, with top_k > 0,
    the [N, top_k] most likely ids in descending order with their log probabilities."""

    logprob: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logprob: Optional[torch.Tensor] = None
    top_id: Optional[torch.Tensor] = None


def _result(out, N: int, top_k: int, dev) -> TokenLogprobs:
    if out:
        r = TokenLogprobs(*(_output(out, k, (N,), torch.float32, dev)
                            for k in ("logprob", "entropy", "lse")))
    else:
        r = TokenLogprobs(*torch.empty((3, N), dtype=torch.float32, device=dev).unbind(0))
    if top_k > 0:
        r.top_logprob = _output(out, "top_logprob", (N, top_k), torch.float32, dev)
        r.top_id = _output(out, "top_id", (N, top_k), torch.int32, dev)
    return r


def _logits(logits, name="logits"):
    """(N, V, row stride) of a [N, V] matrix with unit column stride."""
    if logits.dim() != 2:
        raise ValueError(f"{name} must be [N, V]")
    N, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = logits.stride(0) if N > 1 else V
    if ld < V:
        raise ValueError(f"the rows of {name} overlap")
    return N, V, ld


def token_logprobs(logits, tokens, *, top_k: int = 0, temperature: float = 1.0,
                   ignore_index: int = -100, out: Optional[dict] = None, status=None,
                   stream=None) -> TokenLogprobs:
    """Log probabilities of `tokens` (int32 [N], or None) over logits [N, V] (fp32 or
    bf16, any row stride), with each row's entropy, log-sum-exp and top_k (at most 32)
    most likely ids, via flce_token_logprobs.

    -inf logits are ids that cannot come: never an alternative (missing ones are id -1
    with -inf). `out` may hold preallocated outputs by field name. `status`, an int32
    tensor the caller zeroed, receives device errors (a token out of range, whose log
    probability is NaN)."""
    if out is None and status is None and stream is None:
        r = _fast.token_logprobs(logits, tokens, top_k, temperature, ignore_index)
        if r is not None:
            return TokenLogprobs(*r)
    dev = _device_of(logits, "logits")
    dtype = _dtype_of(logits, "logits")
    N, V, ld = _logits(logits)
    tok = _tokens(tokens, N, dev)
    raw, ctx = _stream(stream, dev)
    with ctx:
        r = _result(out, N, top_k, dev)
    _check(_token_logprobs(logits.data_ptr(), dtype, ld, tok, N, V,
                           _options(ignore_index, top_k, temperature), r.logprob.data_ptr(),
                           r.entropy.data_ptr(), r.lse.data_ptr(), _ptr(r.top_logprob),
                           _ptr(r.top_id), _status(status, dev), raw), "flce_token_logprobs")
    return r


def _upstream(result, N, dev, dlogprob, dentropy, dlse):
    return ([_row_vector(getattr(result, k), N, dev, k) for k in ("logprob", "entropy", "lse")]
            + [_row_vector(g, N, dev, k) for g, k in
               ((dlogprob, "dlogprob"), (dentropy, "dentropy"), (dlse, "dlse"))])


def token_logprobs_backward(logits, tokens, result, *, dlogprob=None, dentropy=None, dlse=None,
                            temperature: float = 1.0, ignore_index: int = -100,
                            in_place: bool = False, out=None, stream=None):
    """Gradient in the logits of a token_logprobs call (`result`), from the upstream
    gradients of its logprob, entropy and lse (fp32 [N], None for 0), via
    flce_token_logprobs_backward. Returns dlogits, of the logits' dtype: `out`, or the
    logits themselves (in_place), or a new tensor, whose rows are at most 15 bytes apart."""
    if out is None and not in_place and stream is None:
        g = _fast.token_logprobs_backward(logits, tokens, result.logprob, result.entropy, result.lse,
                                          dlogprob, dentropy, dlse, temperature, ignore_index)
        if g is not None:
            return g
    dev = _device_of(logits, "logits")
    dtype = _dtype_of(logits, "logits")
    N, V, ld = _logits(logits)
    tok = _tokens(tokens, N, dev)
    raw, ctx = _stream(stream, dev)
    with ctx:
        vecs = _upstream(result, N, dev, dlogprob, dentropy, dlse)
        if in_place:
            grad = logits
        elif out is not None:
            if out.device != dev or out.dtype != logits.dtype or out.shape != logits.shape:
                raise ValueError("out must match the logits' device, dtype and shape")
            grad = out
        else:
            # rows that start relative to 16 bytes as the logits' do (the first one too), however
            # far apart those are
            elt = logits.element_size()
            dld, off = V + (ld - V) % (16 // elt), logits.data_ptr() % 16 // elt
            flat = torch.empty(off + (N - 1) * dld + V if N else 0, dtype=logits.dtype, device=dev)
            grad = flat.as_strided((N, V), (dld, 1), off if N else 0)
    _, _, dld = _logits(grad, "out")
    _check(_token_logprobs_backward(logits.data_ptr(), dtype, ld, tok, N, V,
                                    _options(ignore_index, 0, temperature), *map(_ptr, vecs),
                                    grad.data_ptr(), dld, raw), "flce_token_logprobs_backward")
    return grad


@functools.lru_cache(maxsize=256)
def _linear_ws_bytes(N, D, V, top_k, dw_dtype, backward) -> int:
    size = _size(0)
    o = _options(-100, top_k, 1.0, dw_dtype)
    _check(_linear_ws(N, D, V, o, int(backward), size), "flce_linear_logprobs_workspace_size")
    return int(size.value)


def linear_logprobs_workspace_size(N: int, D: int, V: int, *, top_k: int = 0,
                                   dw_dtype: str = "float32", backward: bool = False) -> int:
    """Workspace bytes of linear_token_logprobs, or of its backward call."""
    return _linear_ws_bytes(N, D, V, 0 if backward else top_k, _dw_code(dw_dtype), backward)


def _dw_code(dw_dtype: str) -> int:
    return {"float32": 0, "bfloat16": 1}[dw_dtype]


def _linear_inputs(H, W):
    dev = _device_of(H, "H")
    _same_device(W, dev, "W")
    if H.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("H and W must be bfloat16")
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1]:
        raise ValueError("H must be [N, D] and W [V, D]")
    if not (H.is_contiguous() and W.is_contiguous()):
        raise ValueError("H and W must be contiguous")
    return dev, H.shape[0], H.shape[1], W.shape[0]


def linear_token_logprobs(H, W, tokens, *, top_k: int = 0, temperature: float = 1.0,
                          ignore_index: int = -100, out: Optional[dict] = None, workspace=None,
                          status=None, timeout_ns: int = 0, stream=None) -> TokenLogprobs:
    """token_logprobs straight from hidden states H (bf16 [N, D]) and the head's weight W
    (bf16 [V, D]), without the [N, V] logits, via flce_linear_token_logprobs."""
    if out is None and workspace is None and status is None and not timeout_ns and stream is None:
        r = _fast.linear_token_logprobs(H, W, tokens, top_k, temperature, ignore_index)
        if r is not None:
            return TokenLogprobs(*r)
    dev, N, D, V = _linear_inputs(H, W)
    tok = _tokens(tokens, N, dev)
    raw, ctx = _stream(stream, dev)
    with ctx:
        r = _result(out, N, top_k, dev)
        ws = _workspace(workspace, _linear_ws_bytes(N, D, V, top_k, 0, False), dev)
    _check(_linear_token_logprobs(H.data_ptr(), W.data_ptr(), tok, N, D, V,
                                  _options(ignore_index, top_k, temperature, 0, timeout_ns),
                                  r.logprob.data_ptr(), r.entropy.data_ptr(), r.lse.data_ptr(),
                                  _ptr(r.top_logprob), _ptr(r.top_id), ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _status(status, dev), raw),
           "flce_linear_token_logprobs")
    return r


def linear_token_logprobs_backward(H, W, tokens, result, *, dlogprob=None, dentropy=None,
                                   dlse=None, temperature: float = 1.0, ignore_index: int = -100,
                                   need_dh: bool = True, need_dw: bool = True,
                                   dw_dtype: str = "float32", out: Optional[dict] = None,
                                   workspace=None, status=None, timeout_ns: int = 0, stream=None):
    """(dH bf16 [N, D], dW fp32 or bf16 [V, D]) of a linear_token_logprobs call, from the
    upstream gradients of its logprob, entropy and lse, via
    flce_linear_token_logprobs_backward. `out` may hold preallocated "dH" and "dW"; one
    that is not needed is None."""
    code = _dw_code(dw_dtype)
    if out is None and workspace is None and status is None and not timeout_ns and stream is None:
        r = _fast.linear_token_logprobs_backward(
            H, W, tokens, result.logprob, result.entropy, result.lse, dlogprob, dentropy, dlse,
            temperature, ignore_index, need_dh, need_dw, code)
        if r is not None:
            return r
    dev, N, D, V = _linear_inputs(H, W)
    tok = _tokens(tokens, N, dev)
    raw, ctx = _stream(stream, dev)
    with ctx:
        vecs = _upstream(result, N, dev, dlogprob, dentropy, dlse)
        dH = _output(out, "dH", (N, D), torch.bfloat16, dev) if need_dh else None
        dW = (_output(out, "dW", (V, D), torch.bfloat16 if code else torch.float32, dev)
              if need_dw else None)
        ws = _workspace(workspace, _linear_ws_bytes(N, D, V, 0, code, True), dev)
    _check(_linear_token_logprobs_backward(H.data_ptr(), W.data_ptr(), tok, N, D, V,
                                           _options(ignore_index, 0, temperature, code, timeout_ns),
                                           *map(_ptr, vecs), _ptr(dH), _ptr(dW), ws.data_ptr(),
                                           ws.numel() * ws.element_size(), _status(status, dev),
                                           raw), "flce_linear_token_logprobs_backward")
    return dH, dW


# ---- layer norm ------------------------------------------------------------------------------


@dataclasses.dataclass
class LayerNormResult:
    """y (x's shape and dtype) and, per row, the fp32 mean and 1 / standard deviation."""

    y: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor


def _norm_rows(x, name):
    """x [..., D] as [N, D] rows of unit column stride: (tensor, N, D, row stride)."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{name} must be [..., D] with D >= 1")
    D = x.shape[-1]
    r = x if x.dim() == 2 else x.reshape(-1, D) if x.numel() else x.new_empty((0, D))
    if D > 1 and r.stride(1) != 1 or r.shape[0] > 1 and r.stride(0) < D:
        r = r.contiguous()
    return r, r.shape[0], D, r.stride(0) if r.shape[0] > 1 else D


def _norm_params(weight, bias, D, dev):
    code = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        _same_device(t, dev, name)
        if t.dim() != 1 or t.shape[0] != D or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [D] tensor")
        c = _dtype_of(t, name)
        if code is not None and c != code:
            raise TypeError("weight and bias must have one dtype")
        code = c
    return code or 0


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, out: Optional[dict] = None,
               stream=None) -> LayerNormResult:
    """Layer norm over the last dimension of x (fp32 or bf16), weight and bias fp32 or
    bf16 (or None), via flce_layer_norm. `out` may hold preallocated "y" (x's shape),
    "mean" and "rstd" ([N])."""
    if out is None and stream is None:
        r = _fast.layer_norm(x, weight, bias, eps)
        if r is not None:
            return LayerNormResult(*r)
    dev = _device_of(x, "x")
    dtype = _dtype_of(x, "x")
    raw, ctx = _stream(stream, dev)
    with ctx:
        r, N, D, ld = _norm_rows(x, "x")
        wcode = _norm_params(weight, bias, D, dev)
        y = _output(out, "y", x.shape, x.dtype, dev)
        if out:
            mean = _output(out, "mean", (N,), torch.float32, dev)
            rstd = _output(out, "rstd", (N,), torch.float32, dev)
        else:
            mean, rstd = torch.empty((2, N), dtype=torch.float32, device=dev).unbind(0)
    _check(_layer_norm(r.data_ptr(), dtype, ld, _ptr(weight), _ptr(bias), wcode, N, D, eps,
                       y.data_ptr(), D, mean.data_ptr(), rstd.data_ptr(), raw), "flce_layer_norm")
    return LayerNormResult(y, mean, rstd)


@functools.lru_cache(maxsize=256)
def _layer_norm_ws_bytes(N, D) -> int:
    size = _size(0)
    _check(_layer_norm_ws(N, D, size), "flce_layer_norm_workspace_size")
    return int(size.value)


def layer_norm_backward(dy, x, weight, result, *, need_dx: bool = True, need_dweight: bool = True,
                        need_dbias: bool = True, out: Optional[dict] = None, workspace=None,
                        stream=None):
    """(dx, dweight, dbias) of a layer_norm call (`result`) via flce_layer_norm_backward;
    dweight and dbias have the weight's dtype (fp32 without a weight). One that is not
    needed is None. `out` may hold preallocated "dx", "dweight" and "dbias"."""
    if out is None and workspace is None and stream is None:
        r = _fast.layer_norm_backward(dy, x, weight, result.mean, result.rstd, need_dx, need_dweight,
                                      need_dbias)
        if r is not None:
            return r
    dev = _device_of(x, "x")
    dtype = _dtype_of(x, "x")
    _same_device(dy, dev, "dy")
    if dy.dtype != x.dtype or dy.shape != x.shape:
        raise ValueError("dy must have x's shape and dtype")
    raw, ctx = _stream(stream, dev)
    with ctx:
        r, N, D, ld = _norm_rows(x, "x")
        g, _, _, ldg = _norm_rows(dy, "dy")
        wcode = _norm_params(weight, None, D, dev)
        mean = _row_vector(result.mean, N, dev, "mean")
        rstd = _row_vector(result.rstd, N, dev, "rstd")
        wtype = weight.dtype if weight is not None else torch.float32
        dx = _output(out, "dx", x.shape, x.dtype, dev) if need_dx else None
        dw = _output(out, "dweight", (D,), wtype, dev) if need_dweight else None
        db = _output(out, "dbias", (D,), wtype, dev) if need_dbias else None
        ws = None
        if need_dweight or need_dbias:
            ws = _workspace(workspace, _layer_norm_ws_bytes(N, D), dev)
    _check(_layer_norm_backward(g.data_ptr(), ldg, r.data_ptr(), dtype, ld, _ptr(weight), wcode,
                                mean.data_ptr(), rstd.data_ptr(), N, D, _ptr(dx), D, _ptr(dw),
                                _ptr(db), _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0,
                                raw), "flce_layer_norm_backward")
    return dx, dw, db


# ---- gradient norm and clipping --------------------------------------------------------------


def _dense(t) -> bool:
    """Whether the tensor's elements fill one block of memory, in some order."""
    if t.is_contiguous():
        return True
    step = 1
    for size, stride in sorted(((s, st) for s, st in zip(t.shape, t.stride()) if s != 1),
                               key=lambda p: p[1]):
        if stride != step:
            return False
        step *= size
    return True


def _clip(grads: list, max_norm: float, outs, norm, workspace, stream):
    if norm is None and workspace is None and stream is None:
        r = _fast.clip_grads(grads, outs, max_norm)
        if r is not None:
            return r
    if outs is not None and outs is not grads and len(outs) != len(grads):
        raise ValueError("out must hold one tensor for each gradient")
    if any(g is None for g in grads):
        there = [i for i, g in enumerate(grads) if g is not None]
        some = [grads[i] for i in there]
        if outs is not None:
            outs = some if outs is grads else [outs[i] for i in there]
        return _clip(some, max_norm, outs, norm, workspace, stream)
    n = len(grads)
    dev = torch.device("cuda", torch.cuda.current_device())
    codes = []
    for g in grads:
        code = _DTYPES.get(g.dtype)
        if code is None:
            raise TypeError(f"gradients must be float32 or bfloat16, not {g.dtype}")
        if g.device != dev:
            raise ValueError(f"every gradient must be on the current CUDA device, {dev}")
        if not g.is_contiguous() and not _dense(g):
            raise ValueError("a gradient must fill its memory without gaps or overlaps")
        codes.append(code)
    if outs is not None and outs is not grads:
        for g, o in zip(grads, outs):
            if o.dtype != g.dtype or o.shape != g.shape or o.device != dev or \
                    (o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous())):
                raise ValueError("out must match the gradients' shapes, strides, dtypes and device")
    raw, ctx = _stream(stream, dev)
    size = _size(0)
    _check(_clip_ws(n, size), "flce_clip_grads_workspace_size")
    with ctx:
        if norm is None:
            norm = torch.empty(1, dtype=torch.float32, device=dev)
        elif norm.device != dev or norm.dtype != torch.float32 or norm.numel() != 1:
            raise ValueError("norm must be a float32 CUDA tensor of one element")
        ws = _workspace(workspace, int(size.value), dev)
    pointers = _vp * n
    src = pointers(*[g.data_ptr() for g in grads])
    dst = None if outs is None else src if outs is grads else pointers(*[o.data_ptr() for o in outs])
    _check(_clip_grads(src, dst, (_i64 * n)(*[g.numel() for g in grads]), (_i32 * n)(*codes), n,
                       max_norm, norm.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                       raw), "flce_clip_grads")
    return norm


def grad_norm(grads: Sequence, *, norm=None, workspace=None, stream=None):
    """The 2-norm over all elements of the gradients (fp32 and bf16 CUDA tensors; a None, of a
    parameter without a gradient, counts nothing), as a float32 [1] tensor, via
    flce_clip_grads."""
    return _clip(list(grads), 1.0, None, norm, workspace, stream)


def clip_grads(grads: Sequence, max_norm: float, *, out: Optional[Sequence] = None, norm=None,
               workspace=None, stream=None):
    """Multiplies the gradients by min(1, max_norm / (norm + 1e-6)), norm their global
    2-norm: in place, or into the tensors of `out`. A None among them, of a parameter without a
    gradient, is passed over. Returns the norm before clipping as a float32 [1] tensor.
    Nothing waits for the GPU."""
    grads = list(grads)
    return _clip(grads, float(max_norm), grads if out is None else list(out), norm, workspace, stream)
